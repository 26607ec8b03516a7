// fsdp_muon.cu -- Newton-Schulz orthogonalisation and the Muon step, for
// sm_103a, with a kernel per product; fsdp_team.cu and fsdp_thin.cu have the
// forms for few small and for thin matrices.
//
//   start    one pass over the input: the norm's partial sums; for the Muon
//            step also the fold of the R ranks' gradients and the momentum
//   scale    x = u / (||u||_F + eps), as hi + lo (below)
//   steps x  S = x x^T (or x^T x: the smaller side), P = b S + c S^2 - d I and
//            x = (a + d) x + P x, three products on the tensor cores. S and P are
//            symmetric: only the squares on and above the diagonal are
//            multiplied, and the epilogue stores both triangles.
//   the last product's epilogue writes the result, or updates the master
//
// Numbers: the operands are fp16 (all are at most about 5 in size; 2^-11
// each), sums are fp32, and x itself is carried to 22 bits, so that the linear
// term is hardly rounded: with x kept in fp16 alone, a 512 x 512 gradient of
// rank 16 under 1 % noise comes out 4e-2 off (its small directions grow by a
// per step, and the rounding with them). P is shifted along its diagonal
// (shift_of): 4e-4 to 7e-4 off for that gradient, 8e-4 for a Gaussian one.
//
// x is kept as two fp16 matrices, hi = fp16(x), which is the products' operand
// as well, and lo = fp16(2048 (x - hi)). Beside fp32 it saves a fifth of the
// last product's traffic, and both move by bulk copies through the warps'
// stages, so that no thread loads or stores them: that epilogue was bound by
// shared memory and L1, which the MMAs' operands use as well (the change took
// 48 x 512 x 512 from 365 to 324 us).
//
// What bounds it. Small matrices: the epilogues. Five steps of 48 x 512 x 512
// are 302 to 310 us, of which the tensor cores are busy for a third; each epilogue
// waits for its first unit and its accumulator in turn, and 192 tiles are 2.5
// waves of the 76 CTA pairs. Few small matrices: latency, see the team kernel.
// Large ones: the tensor cores. A Muon step of 14336 x 4096 over 8 ranks is
// 3.0 to 3.1 ms, 4.0 TFLOP and a first pass of 1.8 GB: 1,290 to 1,310 TFLOP/s in
// all, at the clock that the power limit leaves.
#include "fsdp_muon.cuh"

namespace fsdp {
namespace {

using namespace tc;

struct StartParams {
    int m, n, groups;       // groups of 8 columns per row
    int64_t ldx;            // stride of x
    int vec;                // every row of every input starts on 16 bytes
    float *x32;             // [batch][m][ldx]: the Muon step's u
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
        if (kMuon)
            store8(x + r * p.ldx + c, 8, u);
#pragma unroll
        for (int k = 0; k < 8; k++)
            sq += u[k] * u[k];
    }
    sq = block_sum(sq, sh);
    if (threadIdx.x == 0)
        p.partial[z * kMaxParts + blockIdx.x] = sq;
}

// Where u is: fp32 or bf16 rows.
struct Source {
    const void *p;
    int64_t ld, stride;
    int bf16;
};

// Two values as hi + lo / 2048, each pair in one word.
constexpr float kLoScale = 2048.0f;
__device__ __forceinline__ uint32_t high(float a, float b) { return pack_f16(a, b); }
__device__ __forceinline__ uint32_t low(uint32_t hi, float a, float b)
{
    const float2 h = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
    return pack_f16((a - h.x) * kLoScale, (b - h.y) * kLoScale);
}
__device__ __forceinline__ float2 both(uint32_t hi, uint32_t lo)
{
    const float2 h = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
    const float2 l = __half22float2(*reinterpret_cast<const __half2 *>(&lo));
    return make_float2(fmaf(l.x, 1.0f / kLoScale, h.x), fmaf(l.y, 1.0f / kLoScale, h.y));
}

// x = u / (||u||_F + eps); inv[z]: that factor.
__global__ void __launch_bounds__(kStartThreads) scale_kernel(const Source u, uint16_t *hi, uint16_t *lo,
                                                              const float *partial, int parts, float eps, int m, int n,
                                                              int groups, float *inv_out)
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
    const int64_t total = (int64_t)m * groups;
    hi += z * total * 8;
    lo += z * total * 8;
    for (int64_t i = (int64_t)blockIdx.x * kStartThreads + threadIdx.x; i < total; i += (int64_t)gridDim.x * kStartThreads) {
        const int r = (int)((uint64_t)i < 0x80000000u ? (uint32_t)i / (uint32_t)groups : i / groups);
        const int c = (int)(i - (int64_t)r * groups) * 8;
        float v[8];
        load8(u.p, z * u.stride + r * u.ld + c, n - c, u.bf16, v);
        uint4 h, l;
        uint32_t *hw = reinterpret_cast<uint32_t *>(&h), *lw = reinterpret_cast<uint32_t *>(&l);
#pragma unroll
        for (int k = 0; k < 4; k++) {
            hw[k] = high(v[2 * k] * inv, v[2 * k + 1] * inv);
            lw[k] = low(hw[k], v[2 * k] * inv, v[2 * k + 1] * inv);
        }
        *reinterpret_cast<uint4 *>(hi + i * 8) = h;
        *reinterpret_cast<uint4 *>(lo + i * 8) = l;
    }
}

// S, or (kPoly) P = b S + c S^2 - d I, in fp16; both triangles where one is
// multiplied. Strides are multiples of 16, so groups of 8 and pairs of rows
// stay inside a padded row.
template <bool kPoly>
struct SquareEpi : EpiDefaults {
    static constexpr int kStages = kPoly ? 2 : 1;
    struct Params {
        uint16_t *out;
        int64_t ld, stride;
        float b, c;
        float *trace;          // [batch][groups], of S
        int groups;
    };
    struct Pre {
        float shift;
    };
    static __device__ __forceinline__ void fetch(const Params &p, const Slot &x, int unit, Pre &pre, const EpiMaps &maps)
    {
        if (!kPoly)
            return;
        pre.shift = shift_of(p.trace + x.z * p.groups, x.M, p.b, p.c, x.lane);
        if (unit < x.units())
            x.load_units(&maps.m[1], 1, 1, 0, unit);
    }
    static __device__ __forceinline__ void run(const Params &p, const Slot &x, Pre &pre, const EpiMaps &maps)
    {
        uint16_t *out = p.out + x.z * p.stride;
#pragma unroll 1
        for (int u = x.part; u < x.units(); u += kParts) {
            uint4 own[kPoly ? 8 : 1];  // the thread's own row of the unit of S
            if (kPoly) {
                if (!x.units_loaded(0))
                    return;
#pragma unroll
                for (int i = 0; i < 8; i++)
                    own[kPoly ? i : 0] = *x.piece(x.lane, i, 1);
                __syncwarp();
                if (u + kParts < x.units())
                    x.load_units(&maps.m[1], 1, 1, 0, u + kParts);
            }
            auto finish = [&](int h, float(&v)[32]) {
                x.load_sum(u * 2 + h, v);
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
            x.emit_map<false>(maps.m, u, finish);
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

// x = (a + d) x + (P x). What becomes of it:
//   kKeep    the next step's hi and lo
//   kOut     the result, in bf16
//   kMaster  w = w decay - lr x, and the bf16 parameter
// Maps: hi, lo, and (kKeep) the next hi; lo is updated in place.
enum class Then { kKeep, kOut, kMaster };

struct StepParams {
    float a, b, c;
    const float *trace;
    int groups, k;
    uint16_t *out;
    int64_t ldo, out_stride, n;
    float decay, lr;
    float *master[kMuonMaxMats];
    uint16_t *param[kMuonMaxMats];
};

//
// kSlots: units of hi and lo that a warp has under way. Two take 64 KB from
// the operands' ring, which a long K needs: taken where the epilogue is the
// longer part. One and two: 48 x 512 x 512 312 and 304 us, 16 x 768 x 768 267
// and 261, 16 x 1024 x 1024 472 and 494, 4096 x 14336 2,480 and 2,785.
constexpr int kShortK = 768;
template <Then kThen, int kSlots = 1>
struct StepEpi : EpiDefaults {
    static constexpr int kStages = 2 * kSlots;
    using Params = StepParams;
    struct Pre {
        float a;
    };
    static __device__ __forceinline__ void fetch(const Params &p, const Slot &x, int unit, Pre &pre, const EpiMaps &maps)
    {
        pre.a = p.a + shift_of(p.trace + x.z * p.groups, p.k, p.b, p.c, x.lane);
        x.stage_free();
#pragma unroll
        for (int i = 0; i < kSlots; i++)
            if (unit + i * kParts < x.units())
                x.load_units(maps.m, 2, 2 * i, i, unit + i * kParts);
    }
    static __device__ __forceinline__ void run(const Params &p, const Slot &x, Pre &pre, const EpiMaps &maps)
    {
        const int rows = x.M - x.group_row(0);
#pragma unroll 1
        for (int u = x.part; u < x.units(); u += kParts) {
            const int i = (u - x.part) / kParts, slot = i % kSlots;
            if (i >= kSlots) {
                x.stage_free();
                x.load_units(maps.m, 2, 2 * slot, slot, u);
            }
            if (!x.units_loaded(slot))
                return;
            // The thread's own row of the unit. Where the first stage is
            // needed for what leaves, hi is taken out of it before.
            uint4 hi[8];
            if (kThen != Then::kKeep) {
#pragma unroll
                for (int i = 0; i < 8; i++)
                    hi[i] = *x.piece(x.lane, i, 0);
                __syncwarp();
            }
            auto finish = [&](int h, float(&v)[32]) {
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const uint4 a = kThen != Then::kKeep ? hi[h * 4 + i] : *x.piece(x.lane, h * 4 + i, 2 * slot);
                    const uint4 b = *x.piece(x.lane, h * 4 + i, 2 * slot + 1);
                    const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
                    for (int k = 0; k < 4; k++) {
                        const float2 old = both(aw[k], bw[k]);
                        v[8 * i + 2 * k] = fmaf(pre.a, old.x, v[8 * i + 2 * k]);
                        v[8 * i + 2 * k + 1] = fmaf(pre.a, old.y, v[8 * i + 2 * k + 1]);
                    }
                }
            };
            if (kThen == Then::kKeep) {
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    float v[32];
                    x.load(u * 2 + h, v);
                    finish(h, v);
#pragma unroll
                    for (int g = 0; g < 4; g++) {
                        uint32_t a[4], b[4];
#pragma unroll
                        for (int i = 0; i < 4; i++) {
                            a[i] = high(v[8 * g + 2 * i], v[8 * g + 2 * i + 1]);
                            b[i] = low(a[i], v[8 * g + 2 * i], v[8 * g + 2 * i + 1]);
                        }
                        *x.piece(x.lane, h * 4 + g, 2 * slot) = make_uint4(a[0], a[1], a[2], a[3]);
                        *x.piece(x.lane, h * 4 + g, 2 * slot + 1) = make_uint4(b[0], b[1], b[2], b[3]);
                    }
                }
                x.store_units(&maps.m[2], &maps.m[1], 2 * slot, u);
            } else if (kThen == Then::kOut) {
                const int left = x.N - x.unit_col(u);
                uint16_t *to = p.out + x.z * p.out_stride + x.group_row(0) * p.ldo + x.unit_col(u);
                auto result = [&](int h, float(&v)[32]) {
                    x.load(u * 2 + h, v);
                    finish(h, v);
                };
                if (rows_of_16(p.out, p.ldo | p.out_stride))
                    x.emit16<true>(u, finish, [&](int i, const uint4 &e) {
                        if (i * 4 < rows)
                            put8_16(to + i * 4 * p.ldo, e, left);
                    });
                else
                    x.emit_rows<true>(u, result, [&](int r) {
                        const int64_t row = x.row - x.lane + r;
                        return row < x.M ? p.out + x.z * p.out_stride + row * p.ldo + x.col + u * 64 : nullptr;
                    });
            } else {
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    const int left = x.N - x.group_col(u * 2 + h);
                    const int64_t to = x.group_row(0) * p.n + x.group_col(u * 2 + h);
                    float mine[32], w[8][4];
                    x.load(u * 2 + h, mine);
                    finish(h, mine);
                    auto read_master = [&] {
#pragma unroll
                        for (int i = 0; i < 8; i++)
                            if (i * 4 < rows && left > 0)
                                get4_f32(p.master[x.z] + to + i * 4 * p.n, w[i], left);
                    };
                    x.spread(mine, [&](int i, float(&v)[4]) {
                        if (i * 4 >= rows || left <= 0)
                            return;
#pragma unroll
                        for (int k = 0; k < 4; k++)
                            v[k] = fmaf(-p.lr, v[k], w[i][k] * p.decay);
                        put4_f32(p.master[x.z] + to + i * 4 * p.n, v, left);
                        if (p.param[x.z])
                            put4_16<true>(p.param[x.z] + to + i * 4 * p.n, v, left);
                    }, read_master);
                }
            }
        }
    }
};

// steps = 0: the scaled input is the result.
struct FinishParams {
    Source u;
    const float *inv;
    int m, n;
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
    for (int64_t i = (int64_t)blockIdx.x * kStartThreads + threadIdx.x; i < (int64_t)p.m * p.n;
         i += (int64_t)gridDim.x * kStartThreads) {
        const int64_t r = i / p.n, c = i - r * p.n;
        const int64_t at = z * p.u.stride + r * p.u.ld + c;
        const float v = (p.u.bf16 ? bf16_at(static_cast<const uint16_t *>(p.u.p) + at)
                                  : static_cast<const float *>(p.u.p)[at]) * p.inv[z];
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

int64_t schulz_workspace(int64_t batch, int64_t m, int64_t n, bool muon)
{
    return schulz_plan(batch, m, n, muon, nullptr).bytes;
}

fsdp_status launch_newton_schulz(const SchulzArgs &a, void *workspace, int dev, void *stream)
{
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool muon = a.grads != nullptr;
    const int sms = device_sms(dev);
    const int64_t thin = thin_clocks(a, sms), team = team_clocks(a, dev), products = product_clocks(a, sms);
    const int64_t other = team >= 0 && team < products ? team : products;
    // preferred up to twice the other's estimate, for the sake of fp32: with
    // few rows, fp16 operands leave a nearly low-rank result 8e-3 off (5 x
    // 30011). Where the other is shorter, that costs up to 1.8 times its time
    // (us, here and there: 2 x 6000 x 13 198 and 110, 8 x 24 x 2048 148 and 97,
    // 2 x 8 x 14000 172 and 129)
    if (thin >= 0 && thin < 2 * other)
        return launch_thin(a, workspace, dev, stream);
    if (other == team)
        return launch_team(a, workspace, dev, stream);
    const SchulzPlan q = schulz_plan(a.batch, a.m, a.n, muon, workspace);
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
    const Source u = muon ? Source{q.x32, q.ldx, a.m * q.ldx, 0}
                          : Source{a.g, a.ldg, a.g_stride, a.dtype == FSDP_BF16};
    if ((st = launch("newton_schulz (scale)", scale_kernel, grid, kStartThreads, 0, s, 1, u, q.x16[0], q.lo, q.partial,
                     parts, a.eps, m, n, sp.groups, q.inv)) != FSDP_OK)
        return st;

    if (a.steps == 0) {
        FinishParams fp{};
        fp.u = u;
        fp.inv = q.inv;
        fp.m = m;
        fp.n = n;
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
        const typename SquareEpi<false>::Params e1{q.s, q.ldk, ks, 0.0f, 0.0f, q.trace, (int)q.groups};
        const typename SquareEpi<true>::Params e2{q.p, q.ldk, ks, a.b, a.c, q.trace, (int)q.groups};
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
                                                         &poly, &gram)) != FSDP_OK)
            return st;
        Shape up{};
        up.M = m;
        up.N = n;
        up.K = (int)q.k;
        up.batch = batch;
        up.epi_bytes = kStepBytes;
        const Operand lo{q.lo, a.n, a.m, q.ldx, xs}, next{q.x16[(step + 1) % 2], a.n, a.m, q.ldx, xs};
        auto update = [&](auto epi) {
            using E = decltype(epi);
            // wide: P x, x with its columns adjacent; tall: x P, P symmetric
            return wide ? product<false, true, E>(up, poly, x, false, ep, dev, s, "newton_schulz (x)", &x, &lo, &next)
                        : product<false, false, E>(up, x, poly, false, ep, dev, s, "newton_schulz (x)", &x, &lo, &next);
        };
        st = step + 1 < a.steps ? (q.k <= kShortK ? update(StepEpi<Then::kKeep, 2>{}) : update(StepEpi<Then::kKeep>{}))
             : muon             ? update(StepEpi<Then::kMaster>{})
                                : update(StepEpi<Then::kOut>{});
        if (st != FSDP_OK)
            return st;
    }
    return FSDP_OK;
}

cudaError_t muon_wait_timeouts(unsigned long long *n) { return wait::wait_timeouts(n); }

}  // namespace fsdp
