// fsdp_team.cu -- the Newton-Schulz iteration of matrices that a team of
// blocks holds whole, in one kernel, for sm_103a.
//
// A 512 x 512 product is 2 us of tensor-core time, and a kernel for each of
// the 15 products costs twice that in starting, filling and ending. Here a
// team of blocks, one per 128 x TN tile of x, takes a matrix through all of
// them and then the next one. Its x tile stays in tensor memory in fp32 beside
// the accumulator; S, P and x in fp16 go through global memory (L2), where
// the other blocks' TMA copies read them. After each product the team meets at
// a counter: the writers' stores, a fence to the asynchronous proxy, one
// atomic add per block; the warp that issues the copies waits for the sum.
// All blocks are resident (cooperative launch, one per multiprocessor) and
// every wait is bounded.
//
//   per matrix: read the gradients (and the momentum), sum of squares -- meet
//               -- scale, x16 -- meet -- (S -- meet -- P -- meet -- x -- meet)
//               x steps; the last x goes out instead
//
// 4 x 512 x 512, a Muon step over 4 ranks: 88 us (when first written 95,
// and 104 with a kernel for each product). It is bound by latency: a product is about 0.7 us of waiting for the
// meeting, 0.5 until its first operands are there, 1.7 to 2.2 of products,
// 0.7 of epilogue and 0.6 of meeting, 15 times.
#include "fsdp_muon.cuh"

namespace fsdp {
namespace {

struct TeamParams {
    int m, n, k, wide;
    int batch, teams, size;  // size: blocks of a team
    int x_cols, k_rows, k_cols;  // tiles along the columns of x, and of S
    int steps, bf16, vec;
    float eps, a, b, c;
    int64_t ldx, xs, ldk, ks;
    uint16_t *x16[2], *s, *p;
    float *partial, *trace;
    int groups;  // of 32 rows of S
    unsigned *arrived;
    // newton_schulz
    const void *g;
    int64_t ldg, g_stride;
    uint16_t *out;
    int64_t ldo, out_stride;
    // muon
    int R, nesterov;
    float inv_r, mu, decay, lr;
    float *momentum[kMuonMaxMats];
    float *master[kMuonMaxMats];
    uint16_t *param[kMuonMaxMats];
    const void *grads[kMuonMaxGrads];
};

constexpr int kEpiThreads = 32 * kEpiWarps;

__device__ __forceinline__ void epi_sync()
{
    asm volatile("bar.sync 1, %0;" ::"n"(kEpiThreads) : "memory");
}
// Whether any epilogue thread of the block says so: one answer for all.
__device__ __forceinline__ bool epi_any(bool mine)
{
    uint32_t any;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "bar.red.or.pred q, 1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(any)
        : "r"((uint32_t)mine), "n"(kEpiThreads)
        : "memory");
    return any != 0;
}
// The team's counter reaches `target` within the bounded wait.
__device__ __forceinline__ bool team_wait(const unsigned *arrived, unsigned target)
{
    const uint64_t t0 = now_ns();
    for (uint32_t round = 0; round < (1u << 26); round++) {
        unsigned v;
        asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(arrived) : "memory");
        if (v >= target)
            return true;
        if (round % 64 == 63 && now_ns() - t0 > kWaitNs)
            return false;
    }
    return false;
}
__device__ __forceinline__ void async_fence() { asm volatile("fence.proxy.async.global;" ::: "memory"); }

// 4 elements of a row, `left` of them inside it.
__device__ __forceinline__ void load4(const void *base, int64_t at, int left, bool bf16, bool vec, float (&v)[4])
{
    if (bf16) {
        const uint16_t *p = static_cast<const uint16_t *>(base) + at;
        if (vec && left >= 4) {
            const uint2 u = *reinterpret_cast<const uint2 *>(p);
            v[0] = __uint_as_float(u.x << 16), v[1] = __uint_as_float(u.x & 0xffff0000u);
            v[2] = __uint_as_float(u.y << 16), v[3] = __uint_as_float(u.y & 0xffff0000u);
        } else {
#pragma unroll
            for (int i = 0; i < 4; i++)
                v[i] = i < left ? bf16_at(p + i) : 0.0f;
        }
    } else {
        get4_f32(static_cast<const float *>(base) + at, v, left);
    }
}

// The two operands of a product, as boxes of 64 x 64.
struct Side {
    const CUtensorMap *map;
    bool mn;  // its rows are adjacent, not K
};
template <int kRows>
__device__ __forceinline__ void load_side(unsigned char *dst, const Side &o, int row, int k, int z, uint64_t *bar)
{
#pragma unroll
    for (int i = 0; i < kRows / 64; i++)
        tma_load<1>(dst + i * 8192, o.map, o.mn ? row + i * 64 : k, o.mn ? k : row + i * 64, z, bar);
}

template <int TN, bool kMuon>
__global__ void __launch_bounds__(tc::kThreads, 1)
    team_kernel(const __grid_constant__ CUtensorMap map_x0, const __grid_constant__ CUtensorMap map_x1,
                const __grid_constant__ CUtensorMap map_s, const __grid_constant__ CUtensorMap map_p,
                const __grid_constant__ TeamParams q)
{
    using R = Ring<1, TN>;
    extern __shared__ unsigned char raw[];
    __shared__ float sums[kEpiWarps];
    unsigned char *ring = raw + ((1024 - (saddr(raw) & 1023)) & 1023);
    unsigned char *epi = ring + R::kStages * R::kStageBytes;
    uint64_t *full = reinterpret_cast<uint64_t *>(epi + R::kEpiBytes);
    uint64_t *empty = full + R::kStages;
    uint64_t *acc_full = empty + R::kStages;
    uint32_t *tmem_at = reinterpret_cast<uint32_t *>(acc_full + 4);

    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int team = blockIdx.x / q.size, member = blockIdx.x % q.size;
    const int x_row = member / q.x_cols * kTM, x_col = member % q.x_cols * TN;
    const bool has_k = member < q.k_rows * q.k_cols;
    const int k_row = member / q.k_cols * kTM, k_col = member % q.k_cols * TN;
    unsigned *arrived = q.arrived + team;
    // meetings of one matrix: after the norm, after x16, after each product but the last
    const unsigned meetings = 2 + 3 * q.steps - 1;

    if (warp == 2)
        tmem_alloc<1>(tmem_at, 2 * TN);
    if (threadIdx.x == 0) {
        for (int i = 0; i < R::kStages; i++) {
            bar_init(full + i, 1);
            bar_init(empty + i, 1);
        }
        bar_init(acc_full, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = *tmem_at;
    bool ok = true;

    auto blocks_of = [&](int which) {  // K blocks of S, P, x
        const int K = which == 0 ? (q.wide ? q.n : q.m) : q.k;
        return (K + kBK - 1) / kBK;
    };

    if (warp == 0) {
        int stage = 0;
        uint32_t phase = 0;
        unsigned met = 0;
        for (int z = team; ok && z < q.batch; z += q.teams, met += meetings) {
            for (int t = 0; ok && t < 3 * q.steps; t++) {
                if (!(ok = __all_sync(0xffffffffu, team_wait(arrived, (unsigned)q.size * (met + 2 + t)))))
                    break;
                const int which = t % 3;
                if (which < 2 && !has_k)
                    continue;
                async_fence();
                const CUtensorMap *x = t / 3 % 2 ? &map_x1 : &map_x0;
                const Side a = which == 0   ? Side{x, !q.wide}
                               : which == 1 ? Side{&map_s, false}
                               : q.wide     ? Side{&map_p, false}
                                            : Side{x, false};
                const Side b = which == 0   ? Side{x, !q.wide}
                               : which == 1 ? Side{&map_s, false}
                               : q.wide     ? Side{x, true}
                                            : Side{&map_p, false};
                const int row = which < 2 ? k_row : x_row, col = which < 2 ? k_col : x_col;
                const int nk = blocks_of(which);
                for (int kb = 0; kb < nk; kb++) {
                    if (!(ok = warp_wait(empty + stage, phase ^ 1)))
                        break;
                    if (elect_one()) {
                        bar_expect(full + stage, R::kStageBytes);
                        unsigned char *d = ring + stage * R::kStageBytes;
                        load_side<kTM>(d, a, row, kb * kBK, z, full + stage);
                        load_side<TN>(d + R::kBytesA, b, col, kb * kBK, z, full + stage);
                    }
                    __syncwarp();
                    if (++stage == R::kStages) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
            }
        }
        if (!ok)
            let_copies_land();
    } else if (warp == 1) {
        int stage = 0;
        uint32_t phase = 0;
        for (int z = team; ok && z < q.batch; z += q.teams) {
            for (int t = 0; ok && t < 3 * q.steps; t++) {
                const int which = t % 3;
                if (which < 2 && !has_k)
                    continue;
                const bool a_mn = which == 0 && !q.wide, b_mn = which == 0 ? !q.wide : which == 2 && q.wide;
                const uint32_t idesc = instruction(kTM, TN, false, a_mn, b_mn);
                const uint32_t a_step = k_step(a_mn), b_step = k_step(b_mn);
                const int nk = blocks_of(which);
                for (int kb = 0; kb < nk; kb++) {
                    if (!(ok = warp_wait(full + stage, phase)))
                        break;
                    fence_after();
                    const uint32_t d = saddr(ring + stage * R::kStageBytes);
                    const uint64_t da = operand_desc(d, a_mn), db = operand_desc(d + R::kBytesA, b_mn);
                    if (elect_one()) {
#pragma unroll
                        for (int k = 0; k < kBK / 16; k++)
                            mma_f16<1>(tmem, da + k * a_step, db + k * b_step, idesc, kb > 0 || k > 0);
                        mma_commit<1>(empty + stage);
                    }
                    __syncwarp();
                    if (++stage == R::kStages) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
                if (elect_one())
                    mma_commit<1>(acc_full);
                __syncwarp();
            }
        }
    } else if (warp >= 4) {
        const int quarter = warp % 4, part = (warp - 4) / 4, t0 = threadIdx.x - 128;
        const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
        Slot x{};  // this thread's part of the x tile; the accumulator's columns
        x.row = x_row + quarter * 32 + lane;
        x.col = x_col;
        x.M = q.m;
        x.N = q.n;
        x.lane = lane;
        x.stage = epi + (warp - 4) * 4096;
        x.tmem = tmem + lanes;
        Slot y = x;  // and of the S or P tile
        y.row = k_row + quarter * 32 + lane;
        y.col = k_col;
        y.M = y.N = q.k;
        const uint32_t held = x.tmem + TN;  // x itself, fp32
        uint32_t parity = 0;
        unsigned met = 0;
        // all epilogue threads: what this block wrote is there for the team
        auto meet = [&]() {
            async_fence();
            epi_sync();
            if (t0 == 0)
                asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(arrived) : "memory");
        };
        for (int z = team; z < q.batch; z += q.teams, met += meetings) {
            // ---- input
            float sq = 0.0f;
            const int rows = q.m - x.group_row(0);
#pragma unroll 1
            for (int c = part; c < TN / 32; c += kParts) {
                const int col = x.group_col(c), left = q.n - col;
                float mine[32];
                x.collect(mine, [&](int i, float(&v)[4]) {
                    v[0] = v[1] = v[2] = v[3] = 0.0f;
                    if (i * 4 >= rows || left <= 0)
                        return;
                    const int64_t row = x.group_row(0) + i * 4;
                    if (kMuon) {
                        const int64_t at = row * q.n + col;
                        const void *const *grads = q.grads + z * q.R;
                        load4(grads[0], at, left, q.bf16, q.vec, v);
#pragma unroll 4
                        for (int r = 1; r < q.R; r++) {
                            float o[4];
                            load4(grads[r], at, left, q.bf16, q.vec, o);
#pragma unroll
                            for (int k = 0; k < 4; k++)
                                v[k] = __fadd_rn(v[k], o[k]);
                        }
                        float m[4];
                        get4_f32(q.momentum[z] + at, m, left);
#pragma unroll
                        for (int k = 0; k < 4; k++) {
                            v[k] = __fmul_rn(v[k], q.inv_r);
                            m[k] = fmaf(q.mu, m[k], v[k]);
                            v[k] = q.nesterov ? fmaf(q.mu, m[k], v[k]) : m[k];
                        }
                        put4_f32(q.momentum[z] + at, m, left);
                    } else {
                        load4(q.g, z * q.g_stride + row * q.ldg + col, left, q.bf16, q.vec, v);
                    }
                });
#pragma unroll
                for (int i = 0; i < 32; i++)
                    sq += mine[i] * mine[i];
                tmem_store32(held + c * 32, mine);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                sq += __shfl_xor_sync(0xffffffffu, sq, o);
            if (lane == 0)
                sums[warp - 4] = sq;
            epi_sync();
            if (t0 == 0) {
                float s = sums[0];
                for (int i = 1; i < kEpiWarps; i++)
                    s += sums[i];
                q.partial[z * kMaxParts + member] = s;
            }
            meet();
            // ---- scale
            ok = !epi_any(t0 == 0 && !team_wait(arrived, (unsigned)q.size * (met + 1)));
            if (!ok)
                break;
            sq = 0.0f;
            for (int i = lane; i < q.size; i += 32)
                sq += __ldcg(q.partial + z * kMaxParts + i);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                sq += __shfl_xor_sync(0xffffffffu, sq, o);
            const float inv = 1.0f / (sqrtf(sq) + q.eps);
            auto keep = [&](uint16_t *x16, int c, float(&mine)[32]) {  // the fp16 x
                const int left = q.n - x.group_col(c);
                uint16_t *to = x16 + z * q.xs + x.group_row(0) * q.ldx + x.group_col(c);
                x.spread(mine, [&](int i, float(&v)[4]) {
                    if (i * 4 < rows && left > 0)
                        *reinterpret_cast<uint2 *>(to + i * 4 * q.ldx) = four_16<false>(v);
                });
            };
#pragma unroll 1
            for (int c = part; c < TN / 32; c += kParts) {
                float mine[32];
                __syncwarp();
                tmem_load32(held + c * 32, mine);
#pragma unroll
                for (int i = 0; i < 32; i++)
                    mine[i] *= inv;
                tmem_store32(held + c * 32, mine);
                keep(q.x16[0], c, mine);
            }
            meet();
            // ---- products
            for (int t = 0; t < 3 * q.steps; t++) {
                const int which = t % 3;
                const bool last = t + 1 == 3 * q.steps;
                if (which == 2 || has_k) {
                    uint2 s4[8];  // P: this lane's groups of S, of the first chunk
                    const int yrows = q.k - y.group_row(0);
                    auto fetch_s = [&](int c) {
                        const uint16_t *from = q.s + z * q.ks + y.group_row(0) * q.ldk + y.group_col(c);
#pragma unroll
                        for (int i = 0; i < 8; i++)
                            if (i * 4 < yrows && y.group_col(c) < q.k)
                                s4[i] = *reinterpret_cast<const uint2 *>(from + i * 4 * q.ldk);
                    };
                    if (which == 1 && part < TN / 32)
                        fetch_s(part);
                    // P's shift, while the product runs. S is complete once its
                    // meeting is; x comes a meeting later.
                    const bool diagonal = k_row + quarter * 32 >= k_col && k_row + quarter * 32 < k_col + TN;
                    float shift = 0.0f;
                    bool seen = true;
                    if (which == 1 && diagonal)
                        seen = __all_sync(0xffffffffu, team_wait(arrived, (unsigned)q.size * (met + 2 + t)));
                    if (seen && (which == 2 || (which == 1 && diagonal)))
                        shift = shift_of(q.trace + z * q.groups, q.k, q.b, q.c, lane);
                    ok = !epi_any(!seen || !bar_wait(acc_full, parity));
                    parity ^= 1;
                    if (!ok)
                        break;
                    fence_after();
                    if (which < 2) {
                        uint16_t *out = (which ? q.p : q.s) + z * q.ks;
#pragma unroll 1
                        for (int c = part; c < TN / 32; c += kParts) {
                            if (which == 1 && c > part)
                                fetch_s(c);
                            float mine[32];
                            y.load(c, mine);
                            const bool here = y.col + c * 32 == y.row - lane;  // the diagonal's chunk
                            if (here && which == 0) {
                                const float sum = diagonal_sum(mine, lane);
                                if (lane == 0 && y.row < q.k)
                                    q.trace[z * q.groups + y.row / 32] = sum;
                            }
                            uint16_t *to = out + y.group_row(0) * q.ldk + y.group_col(c);
                            const bool in = y.group_col(c) < q.k;
                            y.spread(mine, [&](int i, float(&v)[4]) {
                                if (i * 4 >= yrows || !in)
                                    return;
                                if (which == 1) {
                                    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&s4[i].x));
                                    const float2 g = __half22float2(*reinterpret_cast<const __half2 *>(&s4[i].y));
                                    v[0] = fmaf(q.c, v[0], q.b * f.x);
                                    v[1] = fmaf(q.c, v[1], q.b * f.y);
                                    v[2] = fmaf(q.c, v[2], q.b * g.x);
                                    v[3] = fmaf(q.c, v[3], q.b * g.y);
                                    if (here) {
#pragma unroll
                                        for (int k = 0; k < 4; k++)
                                            v[k] -= lane % 8 * 4 + k == i * 4 + lane / 8 ? shift : 0.0f;
                                    }
                                }
                                *reinterpret_cast<uint2 *>(to + i * 4 * q.ldk) = four_16<false>(v);
                            });
                        }
                    } else {
#pragma unroll 1
                        for (int c = part; c < TN / 32; c += kParts) {
                            float mine[32], old[32];
                            x.load(c, mine);
                            tmem_load32(held + c * 32, old);
#pragma unroll
                            for (int i = 0; i < 32; i++)
                                mine[i] = fmaf(q.a + shift, old[i], mine[i]);
                            if (!last) {
                                tmem_store32(held + c * 32, mine);
                                keep(q.x16[(t / 3 + 1) % 2], c, mine);
                                continue;
                            }
                            const int col = x.group_col(c), left = q.n - col;
                            x.spread(mine, [&](int i, float(&v)[4]) {
                                if (i * 4 >= rows || left <= 0)
                                    return;
                                const int64_t row = x.group_row(0) + i * 4;
                                if (kMuon) {
                                    const int64_t at = row * q.n + col;
                                    float w[4];
                                    get4_f32(q.master[z] + at, w, left);
#pragma unroll
                                    for (int k = 0; k < 4; k++)
                                        v[k] = fmaf(-q.lr, v[k], w[k] * q.decay);
                                    put4_f32(q.master[z] + at, v, left);
                                    if (q.param[z])
                                        put4_16<true>(q.param[z] + at, v, left);
                                } else {
                                    put4_16<true>(q.out + z * q.out_stride + row * q.ldo + col, v, left);
                                }
                            });
                        }
                    }
                    fence_before();
                } else {
                    // no tile here: the counter takes an arrival of this
                    // meeting only once the one before it is complete
                    ok = !epi_any(t0 == 0 && !team_wait(arrived, (unsigned)q.size * (met + 2 + t)));
                    if (!ok)
                        break;
                }
                if (!last)
                    meet();
            }
            if (!ok)
                break;
        }
    }
    if (!ok && lane == 0)
        atomicAdd(&g_wait_timeouts, 1ull);
    __syncwarp();
    fence_before();
    __syncthreads();
    fence_after();
    if (warp == 2)
        tmem_free<1>(tmem, 2 * TN);
}

struct TeamForm {
    int tn, tiles, teams;
    int64_t clocks;
};

// A meeting and a product's start and end; measured: 512 x 512, 4 matrices.
constexpr int64_t kMeetClocks = 4500;

TeamForm team_form(const SchulzArgs &a, int sms)
{
    const int64_t k = a.m < a.n ? a.m : a.n, l = a.m < a.n ? a.n : a.m;
    TeamForm best{0, 0, 0, 0};
    for (int tn : {256, 128, 64}) {
        const int64_t tiles = (a.m + kTM - 1) / kTM * ((a.n + tn - 1) / tn);
        if (tiles > sms)
            continue;
        const int64_t teams = a.batch < sms / tiles ? a.batch : sms / tiles, rounds = (a.batch + teams - 1) / teams;
        const int64_t nk = (l + kBK - 1) / kBK + 2 * ((k + kBK - 1) / kBK);
        const int64_t t = rounds * a.steps * (nk * block_clocks(1, tn) + 3 * (kMeetClocks + 8 * tn));
        if (best.tn == 0 || t < best.clocks)
            best = {tn, (int)tiles, (int)teams, t};
    }
    return best;
}

template <int TN, bool kMuon>
fsdp_status launch_as(const TeamParams &p, const CUtensorMap (&maps)[4], cudaStream_t stream)
{
    using R = Ring<1, TN>;
    auto kernel = team_kernel<TN, kMuon>;
    cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, R::kSmem);
    if (err != cudaSuccess)
        return set_error(FSDP_ECUDA, "newton_schulz (team): cudaFuncSetAttribute: %s", cudaGetErrorString(err));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.teams * p.size));
    cfg.blockDim = dim3(tc::kThreads);
    cfg.dynamicSmemBytes = R::kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeCooperative;
    at[0].val.cooperative = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    err = cudaLaunchKernelEx(&cfg, kernel, maps[0], maps[1], maps[2], maps[3], p);
    return err == cudaSuccess ? FSDP_OK
                              : set_error(FSDP_ECUDA, "newton_schulz (team) launch failed: %s", cudaGetErrorString(err));
}

}  // namespace

int64_t team_clocks(const SchulzArgs &a, int dev)
{
    if (a.steps < 1)
        return -1;
    const TeamForm f = team_form(a, device_sms(dev));
    return f.tn ? f.clocks : -1;
}

fsdp_status launch_team(const SchulzArgs &a, void *workspace, int dev, void *stream)
{
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const TeamForm f = team_form(a, device_sms(dev));
    const bool muon = a.grads != nullptr;
    const SchulzPlan q = schulz_plan(a.batch, a.m, a.n, muon, workspace);
    TeamParams p{};
    p.m = (int)a.m;
    p.n = (int)a.n;
    p.k = (int)q.k;
    p.wide = a.m <= a.n;
    p.batch = (int)a.batch;
    p.teams = f.teams;
    p.size = f.tiles;
    p.x_cols = (int)((a.n + f.tn - 1) / f.tn);
    p.k_rows = (int)((q.k + kTM - 1) / kTM);
    p.k_cols = (int)((q.k + f.tn - 1) / f.tn);
    p.steps = a.steps;
    p.bf16 = a.dtype == FSDP_BF16;
    p.eps = a.eps, p.a = a.a, p.b = a.b, p.c = a.c;
    p.ldx = q.ldx, p.xs = a.m * q.ldx, p.ldk = q.ldk, p.ks = q.k * q.ldk;
    p.x16[0] = q.x16[0], p.x16[1] = q.x16[1], p.s = q.s, p.p = q.p;
    p.partial = q.partial;
    p.trace = q.trace;
    p.groups = (int)q.groups;
    p.arrived = q.arrived;
    uintptr_t low = 0;  // of every row's start
    if (muon) {
        p.R = a.R;
        p.nesterov = a.nesterov;
        p.inv_r = 1.0f / (float)a.R;
        p.mu = a.mu, p.decay = a.decay, p.lr = a.lr;
        for (int i = 0; i < p.batch; i++) {
            p.momentum[i] = a.momentum[i];
            p.master[i] = a.master[i];
            p.param[i] = a.param_out ? static_cast<uint16_t *>(a.param_out[i]) : nullptr;
        }
        low = (uintptr_t)(a.n * (p.bf16 ? 2 : 4));
        for (int i = 0; i < p.batch * a.R; i++) {
            p.grads[i] = a.grads[i];
            low |= reinterpret_cast<uintptr_t>(a.grads[i]);
        }
    } else {
        p.g = a.g;
        p.ldg = a.ldg;
        p.g_stride = a.g_stride;
        p.out = static_cast<uint16_t *>(a.out);
        p.ldo = a.ldo;
        p.out_stride = a.out_stride;
        low = reinterpret_cast<uintptr_t>(a.g) | (uintptr_t)((a.ldg | a.g_stride) * (p.bf16 ? 2 : 4));
    }
    p.vec = (low & 7u) == 0;
    if (Record *r = current_record())
        return r->add("%s: team tile %d size %d teams %d rounds %d", muon ? "muon" : "newton_schulz", f.tn, f.tiles, f.teams,
                      (p.batch + f.teams - 1) / f.teams);
    CUtensorMap maps[4];
    const Operand ops[4] = {{q.x16[0], a.n, a.m, q.ldx, p.xs},
                            {q.x16[1], a.n, a.m, q.ldx, p.xs},
                            {q.s, q.k, q.k, q.ldk, p.ks},
                            {q.p, q.k, q.k, q.ldk, p.ks}};
    for (int i = 0; i < 4; i++) {
        const fsdp_status st = make_map(&maps[i], ops[i], p.batch, kBK, false);
        if (st != FSDP_OK)
            return st;
    }
    const cudaError_t err = cudaMemsetAsync(q.arrived, 0, p.teams * sizeof(unsigned), s);
    if (err != cudaSuccess)
        return set_error(FSDP_ECUDA, "newton_schulz (team): %s", cudaGetErrorString(err));
    switch (f.tn) {
    case 64: return muon ? launch_as<64, true>(p, maps, s) : launch_as<64, false>(p, maps, s);
    case 128: return muon ? launch_as<128, true>(p, maps, s) : launch_as<128, false>(p, maps, s);
    default: return muon ? launch_as<256, true>(p, maps, s) : launch_as<256, false>(p, maps, s);
    }
}

cudaError_t team_wait_timeouts(unsigned long long *n) { return wait::wait_timeouts(n); }

}  // namespace fsdp
