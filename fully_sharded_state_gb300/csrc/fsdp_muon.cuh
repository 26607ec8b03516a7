// fsdp_muon.cuh -- what the forms of the Newton-Schulz iteration share
// (fsdp_muon.cu, fsdp_team.cu, fsdp_thin.cu): the workspace and the reading of gradients.
#pragma once

#include "fsdp_tc.cuh"

namespace fsdp {

// One kernel for all products of small matrices (fsdp_team.cu). Estimated
// clocks, or -1 where the matrices do not fit it.
int64_t team_clocks(const SchulzArgs &a, int dev);
fsdp_status launch_team(const SchulzArgs &a, void *workspace, int dev, void *stream);
// One block per matrix, in fp32, for thin ones (fsdp_thin.cu). Likewise.
int64_t thin_clocks(const SchulzArgs &a, int sms);
fsdp_status launch_thin(const SchulzArgs &a, void *workspace, int dev, void *stream);

namespace {

using namespace tc;

constexpr int kStartThreads = 256;
constexpr int kMaxParts = 1024;  // partial sums of one matrix's norm

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

// The shift of P. x' = a x + P x = (a + d) x + (P - d I) x for any d; the
// fp32 x of the first term is exact, the fp16 operands of the second are not,
// so d is taken where P's eigenvalues lie: with mu, the mean of S's, about
// b mu + c mu^2. It halves the result's error for full-rank gradients
// (512 x 512 Gaussian: 1.5e-3 to 8e-4; rank 16 under 1 % noise: 4e-4 to 7e-4).
// trace: the sum of S's diagonal, by groups of 32 rows.
__device__ __forceinline__ float shift_of(const float *trace, int k, float b, float c, int lane)
{
    float s = 0.0f;
    for (int i = lane; i < (k + 31) / 32; i += 32)
        s += __ldcg(trace + i);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        s += __shfl_xor_sync(0xffffffffu, s, o);
    const float mu = s / (float)k;
    return mu * fmaf(c, mu, b);
}
// The diagonal's sum of a chunk whose columns are the warp's rows.
__device__ __forceinline__ float diagonal_sum(const float (&v)[32], int lane)
{
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < 32; j++)
        s = lane == j ? v[j] : s;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
}

// S sums over the matrix's longer side. Where even its smallest tiles (128 x
// 64) leave two thirds of the multiprocessors idle and that side is long, the
// sum is cut in parts (Tiles::choose_splits). What that saves grows with the
// longer side l, what joining the parts costs with the shorter one, k, so a sum
// is cut from l = 56 k on. Five steps, in parts and whole, us: 8 x 13 x 6000 136
// and 197, 4 x 24 x 14000 160 and 331, 1 x 128 x 14000 208 and 317, 1 x 400 x 40000
// 532 and 890; below the bound 1 x 300 x 6001 292 and 201, 4 x 256 x 3000 240 and
// 166. Over 332 shapes the worst that the rule does is a quarter (2 x 14000 x 300,
// 349 in parts, which it does not take, and 433).
constexpr int kSplitRatio = 56;
inline int square_splits(int64_t k, int64_t l, int64_t batch)
{
    const int64_t tiles = (k + 127) / 128 * ((k + 63) / 64) * batch, blocks = (l + kBK - 1) / kBK;
    return tiles <= kSplitSms / 3 && blocks >= 32 && l >= kSplitRatio * k ? (int)(blocks / 4) : 1;
}

// The workspace of one call.
struct SchulzPlan {
    int64_t ldx, ldk, k;
    float *x32, *partial, *inv, *trace;
    int64_t groups;     // of 32 rows of S
    int splits;         // parts of S's sum over the longer side, at most
    int *splits_used;
    float *parts;
    unsigned *arrived;  // of each team
    uint16_t *x16[2], *lo, *s, *p;
    int64_t bytes;
};

inline SchulzPlan schulz_plan(int64_t batch, int64_t m, int64_t n, bool muon, void *base)
{
    SchulzPlan q{};
    q.k = m < n ? m : n;
    q.ldx = ceil_to(n, 16);
    q.ldk = ceil_to(q.k, 16);
    Carver c(base);
    q.partial = c.take<float>(batch * kMaxParts);
    q.inv = c.take<float>(batch);
    q.groups = (q.k + 31) / 32;
    q.trace = c.take<float>(batch * q.groups);
    q.arrived = c.take<unsigned>(kMaxParts);
    if (muon)
        q.x32 = c.take<float>(batch * m * q.ldx);
    q.lo = c.take<uint16_t>(batch * m * q.ldx);
    q.x16[0] = c.take<uint16_t>(batch * m * q.ldx);
    q.x16[1] = c.take<uint16_t>(batch * m * q.ldx);
    q.splits = square_splits(q.k, m < n ? n : m, batch);
    q.splits_used = c.take<int>(1);
    if (q.splits > 1)
        q.parts = c.take<float>(parts_floats(q.ldk, q.splits, batch * q.k));
    q.s = c.take<uint16_t>(batch * q.k * q.ldk);
    q.p = c.take<uint16_t>(batch * q.k * q.ldk);
    q.bytes = c.used();
    return q;
}

// The product S (or P) of k x k matrices over K: one triangle and its mirror
// image, or the whole square. The mirror image is scattered stores, 7 bytes'
// time per element against 3 (S), 9 against 4 (P): it pays where K is long.
constexpr int kStepBytes = 5;
inline Shape square_shape(int64_t k, int64_t K, int64_t batch, int sms, bool poly)
{
    Shape whole{}, half{};
    whole.M = whole.N = (int)k;
    whole.K = (int)K;
    whole.batch = (int)batch;
    whole.square = 1;
    whole.epi_bytes = poly ? 4 : 3;
    half = whole;
    half.sym = 1;
    half.epi_bytes = poly ? 9 : 7;
    return best_form(half, sms, 64).cost < best_form(whole, sms, 64).cost ? half : whole;
}

// Clocks of `steps` steps as one kernel per product: the products' own and,
// for each, a kernel's start and end.
constexpr int64_t kLaunchClocks = 4500;
inline int64_t product_clocks(const SchulzArgs &a, int sms)
{
    const int64_t k = a.m < a.n ? a.m : a.n, l = a.m < a.n ? a.n : a.m;
    Shape up{};
    up.M = (int)a.m;
    up.N = (int)a.n;
    up.K = (int)k;
    up.batch = (int)a.batch;
    up.epi_bytes = kStepBytes;
    const Shape sum = square_shape(k, l, a.batch, sms, false);
    const Form f = best_form(sum, sms, 64);
    int64_t gram = f.cost;
    if (square_splits(k, l, a.batch) > 1)  // spread over the grid, and joined
        gram = f.tiles * f.ctas * ((l + kBK - 1) / kBK) * block_clocks(f.ctas, f.columns) / sms + 2 * kLaunchClocks;
    const int64_t t = gram +
                      best_form(square_shape(k, k, a.batch, sms, true), sms, 64).cost + best_form(up, sms, 64).cost;
    return a.steps * (t + 3 * kLaunchClocks);
}

}  // namespace
}  // namespace fsdp
