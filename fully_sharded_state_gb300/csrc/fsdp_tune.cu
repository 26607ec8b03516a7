// fsdp_tune.cu -- losses for tuning a model from what its tokens cost, with
// their gradients, for sm_103a: the preference loss over pairs of sequences
// and the clipped policy loss with a KL term.
//
// Both read a few numbers per row and write one; ordinary calls are bound by
// the way to memory and back, so as little as possible waits for anything else.
//
// Up to 8192 rows one block does all (small_kernel): its rows stay in
// registers, the sequences' ends in shared memory (1600 rows 7.1 us preference, 8.2
// policy; 1M rows of 1024 sequences 19.2 and 24.6).
//
// More rows are cut into chunks, a warp each, with 256 rows of it (count_kernel) or
// 128 (row_kernel) under way at a time. Sequences begin anywhere, so a chunk's part
// of a sequence is a piece, kept at place (chunk + sequence), which no other piece
// has: one of the two grows from each piece to the next.
//   count_kernel  the pieces: what a sequence's rows sum to, how many count
//   sum_kernel    a warp per pair (or sequence): the pieces joined
//   row_kernel    the rows' weights; policy: also the loss, whose last block
//                 adds the blocks' parts up
//
// Sums over rows are of two fp32 numbers, the second one what the first one's
// roundings left (46 bits; 64-bit additions are 2 a clock here, and the
// functions made of them took 10 us of a call). Every order is fixed: the same
// call gives the same bits every time.
#include <cuda_runtime.h>
#include <math_constants.h>

#include <atomic>
#include <cmath>
#include <cstdint>

#include "fsdp_launch.cuh"

namespace fsdp {
namespace {

constexpr int kThreads = 256;
constexpr int kOneBlock = 1024;          // threads of the single block
constexpr int kPerThread = 8;            // rows of one of its threads; count_kernel: windows of 32 rows that a warp has under way
constexpr int kOneBlockRows = kOneBlock * kPerThread;
constexpr int kOneBlockSequences = 2048;
constexpr int kLists = ((3 * kOneBlockSequences + 1) * 4 + 15) / 16 * 16;  // bytes of their lists

// A sum and what its roundings left, or a number and what fp32 leaves of it.
struct Two {
    float hi, lo;
};

__device__ __forceinline__ Two add(Two a, Two b)
{
    const float s = a.hi + b.hi, t = s - a.hi;
    float e = (a.hi - (s - t)) + (b.hi - t);
    e += a.lo + b.lo;
    e = fabsf(s) < CUDART_INF_F ? e : 0.0f;
    Two r;
    r.hi = s + e;
    r.lo = fabsf(s) < CUDART_INF_F ? e - (r.hi - s) : 0.0f;
    return r;
}
// a times b.
__device__ __forceinline__ Two multiply(Two a, Two b)
{
    Two p;
    p.hi = a.hi * b.hi;
    p.lo = fmaf(a.hi, b.lo, fmaf(a.lo, b.hi, fmaf(a.hi, b.hi, -p.hi)));
    if (!(fabsf(p.hi) < CUDART_INF_F))
        p.lo = 0.0f;
    return p;
}
// One over a whole number below 2^24, or above.
__device__ __forceinline__ Two one_over(int n)
{
    const float d = (float)n, r = 1.0f / d;
    return Two{r, fmaf(-r, d, 1.0f) * r - (float)(n - (int)d) * r * r};
}
// a - b without its rounding.
__device__ __forceinline__ Two difference(float a, float b)
{
    Two d;
    d.hi = a - b;
    const float t = d.hi - a;
    d.lo = (a - (d.hi - t)) - (b + t);
    if (!(fabsf(d.hi) < CUDART_INF_F))
        d.lo = 0.0f;
    return d;
}
__device__ __forceinline__ bool above(Two a, Two b) { return a.hi > b.hi || (a.hi == b.hi && a.lo > b.lo); }

struct TuneParams {
    int rows, sequences;
    int chunk, chunks;    // rows of a chunk; a multiple of 256
    int blocks;           // of count_kernel and row_kernel: entries of `bad` and `counted`
    int seq_blocks;       // of sum_kernel: entries of `filled`
    const float *row_loss, *ref, *old, *advantages;
    const int64_t *offsets;
    const uint8_t *mask;
    float *loss, *row_weights, *margins, *kl, *clipped;
    // workspace
    Two *piece;           // [chunks + sequences]
    int *piece_count;
    int *bad;             // offsets that fall or leave the rows, by block
    int *counted;         // rows that count, by block
    int *filled;          // sequences with such rows, by block
    float *term;          // of a pair
    float *share;         // of a sequence
    Two *part;            // [2][blocks]: loss, KL
    int *part_clipped;
    int *done;
    // numbers
    Two beta;
    float smoothing;
    int average, by_sequence, reduction;
    float low, high;      // 1 - clip_low, 1 + clip_high
    Two log_low, log_high;
    float kl_coef;
};

__device__ __forceinline__ int warp_sum(int v) { return __reduce_add_sync(0xffffffffu, v); }
__device__ __forceinline__ Two warp_sum(Two v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v = add(v, Two{__shfl_xor_sync(0xffffffffu, v.hi, o), __shfl_xor_sync(0xffffffffu, v.lo, o)});
    return v;
}

__device__ __forceinline__ int get(const int *p) { return __ldcg(p); }
__device__ __forceinline__ Two get(const float *p) { return Two{__ldcg(p), 0.0f}; }
__device__ __forceinline__ Two get(const Two *p)
{
    const float2 v = __ldcg(reinterpret_cast<const float2 *>(p));
    return Two{v.x, v.y};
}
__device__ __forceinline__ int add(int a, int b) { return a + b; }
// The sum over the block of each thread's v, for every thread.
template <typename T>
__device__ __forceinline__ T block_add(T v, T *sh)
{
    v = warp_sum(v);
    __syncthreads();
    if (threadIdx.x % 32 == 0)
        sh[threadIdx.x / 32] = v;
    __syncthreads();
    v = (int)threadIdx.x % 32 < (int)blockDim.x / 32 ? sh[threadIdx.x % 32] : T{};
    return warp_sum(v);
}
// And of the n numbers of a list.
template <typename T, typename E>
__device__ __forceinline__ T block_sum(const E *list, int n, T *sh)
{
    T v{};
    for (int i = threadIdx.x; i < n; i += blockDim.x)
        v = add(v, get(list + i));
    return block_add(v, sh);
}

// The sequences around a warp's rows, which rise: 32 of their ends, a lane each.
struct Ends {
    int first;      // lane l has the end of sequence first + l; -1 is what lies before them all
    int end;
    int seq, until; // the last sequence that was asked for, and its end

    __device__ __forceinline__ void load(const TuneParams &p)
    {
        const int i = first + 1 + (int)(threadIdx.x % 32);
        if (i > p.sequences) {
            end = 0x7fffffff;  // no row's
        } else {
            const int64_t v = p.offsets[i];
            end = v < 0 ? 0 : v > p.rows ? p.rows : (int)v;
        }
    }
    // The sequence of `row`, by 32 probes a step.
    __device__ __forceinline__ Ends(const TuneParams &p, int row)
    {
        int lo = 0, hi = p.sequences + 1;  // offsets below lo are at most row, those from hi on above it
        while (lo < hi) {
            const int step = (hi - lo + 31) / 32, i = lo + (int)(threadIdx.x % 32) * step;
            const int k = __popc(__ballot_sync(0xffffffffu, i < hi && p.offsets[min(i, p.sequences)] <= row));
            if (k == 0)
                break;
            hi = min(hi, lo + k * step);
            lo += (k - 1) * step + 1;
        }
        first = lo - 1;
        load(p);
        seq = first;
        until = __shfl_sync(0xffffffffu, end, 0);
    }
    // The sequence of this lane's row, row0 + lane; `sequences` behind the last
    // one. Lanes that are not live get any. A converged warp's.
    __device__ __forceinline__ int at(const TuneParams &p, int row0, bool live)
    {
        if (row0 + 31 < until)
            return seq;
        const int row = row0 + (int)(threadIdx.x % 32);
        int s = 0;
        bool open = live;
        while (true) {
            int c = 0;
            const bool past = __shfl_sync(0xffffffffu, end, 31) <= row;
#pragma unroll
            for (int b = 16; b > 0; b >>= 1)
                c += __shfl_sync(0xffffffffu, end, c + b - 1) <= row ? b : 0;
            c += c == 31 && past ? 1 : 0;
            if (open && c < 32) {
                s = first + c;
                open = false;
            }
            if (!__any_sync(0xffffffffu, open))
                break;
            first += 32;
            load(p);
        }
        const unsigned alive = __ballot_sync(0xffffffffu, live);
        seq = __shfl_sync(0xffffffffu, s, 31 - __clz(alive));
        until = __shfl_sync(0xffffffffu, end, seq - first);
        return s;
    }
};

// -- a row, a pair -----------------------------------------------------------------

// What a row adds to its sequence's sum.
__device__ __forceinline__ Two gain(const TuneParams &p, float row_loss, float ref)
{
    return p.ref ? difference(ref, row_loss) : Two{-row_loss, 0.0f};
}

// A pair's margin, loss and sequences' weights from its sums and counts.
struct Pair {
    float margin, term, good, poor;
};
__device__ __forceinline__ Pair pair_of(const TuneParams &p, Two sg, Two sp, int ng, int np, bool bad)
{
    Pair r;
    const Two wg = p.average ? one_over(max(ng, 1)) : Two{1.0f, 0.0f}, wp = p.average ? one_over(max(np, 1)) : Two{1.0f, 0.0f};
    const Two mean_p = multiply(sp, wp);
    const Two m = multiply(add(multiply(sg, wg), Two{-mean_p.hi, -mean_p.lo}), p.beta);
    r.margin = bad ? CUDART_NAN_F : m.hi + m.lo;
    const float rest = fabsf(r.margin) < 1e30f ? (m.hi - r.margin) + m.lo : 0.0f;
    // e = exp(-|m|), with what rounding m left
    const float size = fabsf(r.margin);
    float e = expf(-size);
    e = fmaf(e, r.margin < 0.0f ? rest : -rest, e);
    const float s = p.smoothing, one = 1.0f + e;
    // softplus(|m|) = |m| + log1p(e), softplus(-|m|) = log1p(e)
    const float soft = log1pf(e);
    const float on = r.margin < 0.0f ? 1.0f - s : s;  // of the softplus that has |m| in it
    r.term = on == 0.0f ? soft : fmaf(on, size, soft);
    if (bad)
        r.term = CUDART_NAN_F;
    // d/dm = s - sigma(-m)
    float slope;
    if (r.margin < 0.0f)
        slope = (s - 1.0f) + e / one;
    else
        slope = s - e / one;
    const float k = p.beta.hi * slope / (p.reduction == FSDP_MEAN ? (float)(p.sequences / 2) : 1.0f);
    r.good = bad ? 0.0f : -k * wg.hi;
    r.poor = bad ? 0.0f : k * wp.hi;
    return r;
}

// Beyond kFar exp(v) is multiplied into a result before it leaves fp32: it is
// taken as exp(v / 2) twice, with the factors between, so that a result is
// infinite only where fp32 does not hold it. (exp(64) is 2^92: up to there
// factors of 2^35 have room.) lo: what rounding left of v.
constexpr float kFar = 64.0f;
__device__ __forceinline__ float far_exp(float v, float lo, float a, float k)
{
    const float half = expf(0.5f * v), r = half * a * k * half;
    return fabsf(r) < CUDART_INF_F ? fmaf(r, lo, r) : r;
}

// KL estimates are summed at 2^-40 of their size, which is exact: the mean of
// 2^31 of them is infinite only where fp32 does not hold it.
constexpr float kKlUnit = 1.0f / (float)(1ull << 40);

// exp(d) - 1 - d up to kFar; its series where the two would cancel.
__device__ __forceinline__ float kl_of(float d, float expm1_d)
{
    if (fabsf(d) >= 0.25f)
        return expm1_d - d;
    float s = 1.0f / 40320.0f;
    s = fmaf(s, d, 1.0f / 5040.0f);
    s = fmaf(s, d, 1.0f / 720.0f);
    s = fmaf(s, d, 1.0f / 120.0f);
    s = fmaf(s, d, 1.0f / 24.0f);
    s = fmaf(s, d, 1.0f / 6.0f);
    s = fmaf(s, d, 0.5f);
    return s * d * d;
}

// A row of the policy loss: its term and its slope, which count k times, its KL
// estimate in kKlUnit.
struct PolicyRow {
    float term, slope, k, kl;
    bool cut;
};
__device__ __forceinline__ PolicyRow policy_row(const TuneParams &p, float now, float old, float ref, float a, float k)
{
    PolicyRow r{0.0f, 0.0f, k, 0.0f, false};
    const Two l = difference(old, now);
    r.cut = a > 0.0f ? above(l, p.log_high) : a < 0.0f && above(p.log_low, l);
    if (a != 0.0f) {
        const float e = expf(l.hi), ratio = fmaf(e, l.lo, e);
        r.term = -(r.cut ? (a > 0.0f ? p.high : p.low) : ratio) * a;
        r.slope = r.cut ? 0.0f : ratio * a;
    }
    float d = 0.0f, g = 0.0f;
    if (p.ref) {
        d = now - ref;
        g = expm1f(d);
        r.kl = kl_of(d, g);
    }
    // without a coefficient the KL is only watched: 0 times an infinite one is no part of the loss
    const float coef = p.kl_coef;
    if (l.hi > kFar || d > kFar) {
        const bool far = l.hi > kFar && a != 0.0f && !r.cut;
        const float ratio = far ? far_exp(l.hi, l.lo, a, k) : 0.0f;
        r.term = far ? -ratio : r.term * k;
        r.slope = far ? ratio : r.slope * k;
        if (coef != 0.0f) {
            const float v = d > kFar ? far_exp(d, 0.0f, coef, k) : 0.0f;
            r.term += d > kFar ? v : coef * r.kl * k;
            r.slope += d > kFar ? v : coef * g * k;
        }
        r.k = 1.0f;
        r.kl = d > kFar ? far_exp(d, 0.0f, kKlUnit, 1.0f) : r.kl * kKlUnit;
    } else {
        if (coef != 0.0f) {
            r.term = fmaf(coef, r.kl, r.term);
            r.slope = fmaf(coef, g, r.slope);
        }
        r.kl *= kKlUnit;
    }
    return r;
}

__device__ __forceinline__ void policy_results(const TuneParams &p, Two loss, Two kl, int clipped, int counted, bool bad)
{
    *p.loss = bad ? CUDART_NAN_F : loss.hi;
    *p.kl = bad ? CUDART_NAN_F : kl.hi / (float)max(counted, 1) / kKlUnit;
    *p.clipped = bad ? CUDART_NAN_F : (float)clipped / (float)max(counted, 1);
}

// What a row's term counts for, but for the sequence's part of it.
__device__ __forceinline__ float row_share(const TuneParams &p, int counted, int filled)
{
    return p.reduction == FSDP_POLICY_MEAN       ? 1.0f / (float)max(counted, 1)
           : p.reduction == FSDP_POLICY_SEQUENCE ? 1.0f / (float)max(filled, 1)
                                                 : 1.0f;
}

__device__ __forceinline__ bool offsets_bad(const TuneParams &p, int64_t i, int64_t step)
{
    bool bad = i == 0 && (p.offsets[0] < 0 || p.offsets[0] > p.rows);
    for (; i < p.sequences; i += step)
        bad |= p.offsets[i] > p.offsets[i + 1] || p.offsets[i + 1] > p.rows;
    return bad;
}

// -- one block ---------------------------------------------------------------------

// Rows tid, tid + 1024, ... are a thread's; their gains are added up from shared
// memory. Counts are whole numbers, whose order is of
// no matter.
template <bool kPreference>
__global__ void __launch_bounds__(kOneBlock) small_kernel(const TuneParams p)
{
    extern __shared__ unsigned char dyn[];
    // [0, sequences]: where they begin and end; the sequences' weights; counts; preference: their sums, the rows' gains
    int *begin = reinterpret_cast<int *>(dyn);
    float *share = reinterpret_cast<float *>(begin + p.sequences + 1);
    int *count = reinterpret_cast<int *>(share + p.sequences);
    float2 *sums = reinterpret_cast<float2 *>(dyn + kLists), *gains = sums + kOneBlockSequences;
    __shared__ Two sh2[32];
    __shared__ int shi[32];
    launch_wait();
    launch_next();
    const int t = threadIdx.x, lane = t % 32, warp = t / 32;
    float now[kPerThread], other[kPerThread], third[kPerThread], adv[kPerThread];
    bool in[kPerThread];
    bool bad = false;
#pragma unroll
    for (int i = 0; i < kPerThread; i++) {
        const int r = i * kOneBlock + t;
        const bool live = r < p.rows;
        now[i] = live ? p.row_loss[r] : 0.0f;
        other[i] = live && !kPreference ? p.old[r] : 0.0f;
        third[i] = live && p.ref ? p.ref[r] : 0.0f;
        adv[i] = live && !kPreference && !p.by_sequence ? p.advantages[r] : 0.0f;
        in[i] = live && (p.mask == nullptr || p.mask[r] != 0);
    }
    if (p.offsets) {
        for (int i = t; i <= p.sequences; i += kOneBlock) {
            const int64_t v = p.offsets[i];
            begin[i] = v < 0 ? 0 : v > p.rows ? p.rows : (int)v;
        }
        for (int i = t; i < p.sequences; i += kOneBlock)
            count[i] = 0;
        bad = offsets_bad(p, t, kOneBlock);
    }
    bad = __syncthreads_or(bad);
    int seq[kPerThread], counted = 0;
#pragma unroll
    for (int i = 0; i < kPerThread; i++) {
        const int r = i * kOneBlock + t;
        int lo = 0;
        if (p.offsets && r < p.rows) {
            int hi = p.sequences + 1;
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (begin[mid] <= r)
                    lo = mid + 1;
                else
                    hi = mid;
            }
            lo--;
            in[i] = in[i] && !bad && lo >= 0 && lo < p.sequences;
        }
        seq[i] = lo;
        counted += in[i];
        if (kPreference && r < p.rows) {
            const Two g = gain(p, now[i], third[i]);
            gains[r] = in[i] ? make_float2(g.hi, g.lo) : make_float2(0.0f, 0.0f);
        }
    }
    if (kPreference) {
        if (p.average) {
#pragma unroll
            for (int i = 0; i < kPerThread; i++)
                if (in[i])
                    atomicAdd(&count[seq[i]], 1);
        }
        __syncthreads();
        // Eight lanes a sequence; a whole warp one of more than 256 rows, of which
        // there are 32 at most. (A warp each, 1358 sequences of two rows took 6 us.)
        auto sum = [&](int s, int from, int step) {
            Two v{0.0f, 0.0f};
            for (int r = begin[s] + from; r < begin[s + 1]; r += step) {
                const float2 g = gains[r];
                v = add(v, Two{g.x, g.y});
            }
            return v;
        };
        constexpr int kShort = 256;
        for (int s0 = warp * 4; s0 < p.sequences && !bad; s0 += kOneBlock / 8) {
            const int s = s0 + lane / 8;
            const bool mine = s < p.sequences && begin[s + 1] - begin[s] <= kShort;
            Two v = mine ? sum(s, lane % 8, 8) : Two{0.0f, 0.0f};
#pragma unroll
            for (int o = 4; o > 0; o >>= 1)
                v = add(v, Two{__shfl_xor_sync(0xffffffffu, v.hi, o), __shfl_xor_sync(0xffffffffu, v.lo, o)});
            if (mine && lane % 8 == 0)
                sums[s] = make_float2(v.hi, v.lo);
        }
        for (int s = warp; s < p.sequences && !bad; s += kOneBlock / 32) {
            if (begin[s + 1] - begin[s] <= kShort)
                continue;
            const Two v = warp_sum(sum(s, lane, 32));
            if (lane == 0)
                sums[s] = make_float2(v.hi, v.lo);
        }
        __syncthreads();
        const int pairs = p.sequences / 2;
        Two loss{0.0f, 0.0f};
        for (int i = t; i < pairs; i += kOneBlock) {
            const float2 g = bad ? make_float2(0.0f, 0.0f) : sums[2 * i], q = bad ? g : sums[2 * i + 1];
            const Pair r = pair_of(p, Two{g.x, g.y}, Two{q.x, q.y}, count[2 * i], count[2 * i + 1], bad);
            p.margins[i] = r.margin;
            share[2 * i] = r.good;
            share[2 * i + 1] = r.poor;
            loss = add(loss, Two{r.term, 0.0f});
        }
        loss = block_add(loss, sh2);  // its barriers stand between the weights and their use
        if (t == 0)
            *p.loss = bad ? CUDART_NAN_F : p.reduction == FSDP_MEAN ? loss.hi / (float)max(pairs, 1) : loss.hi;
#pragma unroll
        for (int i = 0; i < kPerThread; i++) {
            const int r = i * kOneBlock + t;
            if (r < p.rows)
                p.row_weights[r] = in[i] ? share[seq[i]] : 0.0f;
        }
    } else {
        int filled = 0;
        if (p.reduction == FSDP_POLICY_SEQUENCE) {
#pragma unroll
            for (int i = 0; i < kPerThread; i++)
                if (in[i])
                    atomicAdd(&count[seq[i]], 1);
            __syncthreads();
            for (int i = t; i < p.sequences; i += kOneBlock) {
                filled += count[i] > 0;
                share[i] = count[i] > 0 ? 1.0f / (float)count[i] : 0.0f;
            }
            filled = block_add(filled, shi);
        }
        counted = block_add(counted, shi);
        const float per = row_share(p, counted, filled);
        float loss = 0.0f, kl = 0.0f;
        int clipped = 0;
#pragma unroll
        for (int i = 0; i < kPerThread; i++) {
            const int r = i * kOneBlock + t;
            float weight = 0.0f;
            if (in[i]) {
                const float k = p.reduction == FSDP_POLICY_SEQUENCE ? per * share[seq[i]] : per;
                const PolicyRow q = policy_row(p, now[i], other[i], third[i], p.by_sequence ? p.advantages[seq[i]] : adv[i], k);
                weight = q.slope * q.k;
                loss = fmaf(q.term, q.k, loss);
                kl += q.kl;
                clipped += q.cut;
            }
            if (r < p.rows)
                p.row_weights[r] = weight;
        }
        const Two all = block_add(Two{loss, 0.0f}, sh2), all_kl = block_add(Two{kl, 0.0f}, sh2);
        clipped = block_add(clipped, shi);
        if (t == 0)
            policy_results(p, all, all_kl, clipped, counted, bad);
    }
}

// -- the pieces --------------------------------------------------------------------

template <bool kPreference>
__device__ __forceinline__ void count_chunk(const TuneParams &p, int c, int &counted)
{
    const int lane = threadIdx.x % 32, lo = c * p.chunk, hi = p.rows - lo < p.chunk ? p.rows : lo + p.chunk;
    Ends ends(p, lo);
    int open = -1;  // the sequence that `sum` and `n`, a part per lane, are of
    Two sum{0.0f, 0.0f};
    int n = 0;
    auto put = [&](int s, Two v, int k) {
        if (s >= 0 && s < p.sequences) {
            if (kPreference)
                p.piece[c + s] = v;
            p.piece_count[c + s] = k;
        }
    };
    for (int b0 = lo; b0 < hi; b0 += 32 * kPerThread) {
        float now[kPerThread], ref[kPerThread];
        bool in[kPerThread];
#pragma unroll
        for (int i = 0; i < kPerThread; i++) {
            const int r = b0 + i * 32 + lane;
            const bool live = r < hi;
            now[i] = kPreference && live ? p.row_loss[r] : 0.0f;
            ref[i] = kPreference && live && p.ref ? p.ref[r] : 0.0f;
            in[i] = live && (p.mask == nullptr || p.mask[r] != 0);
        }
#pragma unroll
        for (int i = 0; i < kPerThread; i++) {
            const int r0 = b0 + i * 32;
            if (r0 >= hi)
                break;
            const bool live = r0 + lane < hi;
            const int s = ends.at(p, r0, live);
            const bool one = in[i] && s >= 0 && s < p.sequences;
            Two v = kPreference && one ? gain(p, now[i], ref[i]) : Two{0.0f, 0.0f};
            counted += one;
            if (__all_sync(0xffffffffu, s == open || !live)) {
                sum = add(sum, v);
                n += one;
                continue;
            }
            // the open sequence ends here, others may begin and end
            const bool mine = s == open && live;
            if (kPreference) {
                const Two all = warp_sum(mine ? add(sum, v) : sum);
                const int all_n = warp_sum(n + (mine ? (int)one : 0));
                if (lane == 0)
                    put(open, all, all_n);
            } else {
                const int all_n = warp_sum(n + (mine ? (int)one : 0));
                if (lane == 0)
                    put(open, v, all_n);
            }
            // sums from each sequence's first lane on
            int k = one;
#pragma unroll
            for (int o = 1; o < 32; o *= 2) {
                const int wk = __shfl_up_sync(0xffffffffu, k, o), ws = __shfl_up_sync(0xffffffffu, s, o);
                const bool same = lane >= o && ws == s;
                if (kPreference) {
                    const Two w{__shfl_up_sync(0xffffffffu, v.hi, o), __shfl_up_sync(0xffffffffu, v.lo, o)};
                    v = same ? add(v, w) : v;
                }
                k += same ? wk : 0;
            }
            const int next = __shfl_down_sync(0xffffffffu, s, 1);
            const int last = 31 - __clz(__ballot_sync(0xffffffffu, live));
            if (live && !mine && lane < last && next != s)
                put(s, v, k);
            open = ends.seq;
            sum = lane == last ? v : Two{0.0f, 0.0f};
            n = lane == last ? k : 0;
        }
    }
    const Two all = kPreference ? warp_sum(sum) : sum;
    const int all_n = warp_sum(n);
    if (lane == 0)
        put(open, all, all_n);
}

template <bool kPreference>
__global__ void __launch_bounds__(kThreads) count_kernel(const TuneParams p)
{
    __shared__ int shi[32];
    launch_wait();
    launch_next();
    const int block = blockIdx.x, blocks = gridDim.x, warps = kThreads / 32;
    int counted = 0;
    for (int c = block * warps + (int)threadIdx.x / 32; c < p.chunks; c += blocks * warps) {
        if (p.offsets) {
            count_chunk<kPreference>(p, c, counted);
        } else {
            const int lo = c * p.chunk, hi = p.rows - lo < p.chunk ? p.rows : lo + p.chunk;
#pragma unroll 8
            for (int r = lo + (int)threadIdx.x % 32; r < hi; r += 32)
                counted += p.mask == nullptr || p.mask[r] != 0;
        }
    }
    const bool bad = __syncthreads_or(
        p.offsets && offsets_bad(p, (int64_t)block * kThreads + threadIdx.x, (int64_t)blocks * kThreads));
    counted = block_add(counted, shi);
    if (threadIdx.x == 0) {
        p.counted[block] = counted;
        p.bad[block] = bad;
        if (block == 0)
            *p.done = 0;
    }
}

__device__ __forceinline__ bool any_bad(const TuneParams &p)
{
    bool bad = false;
    for (int i = threadIdx.x; i < p.blocks; i += blockDim.x)
        bad |= __ldcg(p.bad + i) != 0;
    return __syncthreads_or(bad) != 0;
}

// -- the sequences -----------------------------------------------------------------

// The pieces of sequence s, by a warp.
template <bool kSums>
__device__ __forceinline__ void join(const TuneParams &p, int s, Two &sum, int &n)
{
    const int lo = (int)p.offsets[s], hi = (int)p.offsets[s + 1], lane = threadIdx.x % 32;
    sum = Two{0.0f, 0.0f};
    int k = 0;
    if (lo < hi) {
        const int last = (hi - 1) / p.chunk;
        for (int c = lo / p.chunk + lane; c <= last; c += 32) {
            if (kSums)
                sum = add(sum, get(p.piece + c + s));
            k += __ldcg(p.piece_count + c + s);
        }
    }
    if (kSums)
        sum = warp_sum(sum);
    n = warp_sum(k);
}

// The last block to come here, of all of a launch's.
__device__ __forceinline__ bool last_block(const TuneParams &p, bool *last)
{
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        *last = atomicAdd(p.done, 1) == (int)gridDim.x - 1;
        __threadfence();
    }
    __syncthreads();
    return *last;
}

// Preference: margins, the sequences' weights, the losses, which the last
// block adds up. Policy, the mean of means: one over the sequences' counts,
// and how many have rows.
template <bool kPreference>
__global__ void __launch_bounds__(kThreads) sum_kernel(const TuneParams p)
{
    __shared__ Two sh2[32];
    __shared__ int shi[32];
    __shared__ bool last;
    launch_wait();
    launch_next();
    const bool bad = any_bad(p);
    const int warps = kThreads / 32, warp = threadIdx.x / 32, lane = threadIdx.x % 32, pairs = p.sequences / 2;
    int filled = 0;
    for (int i = blockIdx.x * warps + warp; i < (kPreference ? pairs : p.sequences); i += gridDim.x * warps) {
        Two s[2] = {};
        int n[2] = {};
        if (kPreference) {
            for (int j = 0; j < 2 && !bad; j++)
                join<true>(p, 2 * i + j, s[j], n[j]);
            const Pair q = pair_of(p, s[0], s[1], n[0], n[1], bad);
            if (lane == 0) {
                p.margins[i] = q.margin;
                p.term[i] = q.term;
                p.share[2 * i] = q.good;
                p.share[2 * i + 1] = q.poor;
            }
        } else {
            if (!bad)
                join<false>(p, i, s[0], n[0]);
            filled += lane == 0 && n[0] > 0;
            if (lane == 0)
                p.share[i] = n[0] > 0 ? 1.0f / (float)n[0] : 0.0f;
        }
    }
    if (kPreference) {
        if (!last_block(p, &last))
            return;
        const Two sum = block_sum(p.term, pairs, sh2);
        if (threadIdx.x == 0)
            *p.loss = bad ? CUDART_NAN_F : p.reduction == FSDP_MEAN ? sum.hi / (float)max(pairs, 1) : sum.hi;
    } else {
        filled = block_add(filled, shi);
        if (threadIdx.x == 0)
            p.filled[blockIdx.x] = filled;
    }
}

// -- the rows --------------------------------------------------------------------

// Windows of 32 rows that a warp has under way. Few: their code is run once a
// warp, and fetching that of eight takes longer than the rows (1M rows, 1024
// sequences, all three kernels: 30.9 us with 8, 25.5 with 4, 27.1 with 2).
constexpr int kRowFlight = 4;

template <bool kPreference>
__global__ void __launch_bounds__(kThreads) row_kernel(const TuneParams p)
{
    __shared__ Two sh2[32];
    __shared__ int shi[32];
    __shared__ bool last;
    launch_wait();
    launch_next();
    const int block = blockIdx.x, blocks = gridDim.x, warps = kThreads / 32, lane = threadIdx.x % 32;
    bool bad = false;
    int counted = 0, filled = 0;
    float per = 1.0f;
    if (!kPreference) {
        // the preference loss has weights of 0 in this case
        bad = any_bad(p);
        counted = block_sum(p.counted, p.blocks, shi);
        if (p.reduction == FSDP_POLICY_SEQUENCE)
            filled = block_sum(p.filled, p.seq_blocks, shi);
        per = row_share(p, counted, filled);
    }
    Two loss{0.0f, 0.0f}, kl{0.0f, 0.0f};
    int clipped = 0;
    for (int c = block * warps + (int)threadIdx.x / 32; c < p.chunks; c += blocks * warps) {
        const int lo = c * p.chunk, hi = p.rows - lo < p.chunk ? p.rows : lo + p.chunk;
        auto chunk = [&](auto sequence) {
#pragma unroll 1
            for (int b0 = lo; b0 < hi; b0 += 32 * kRowFlight) {
                float now[kRowFlight], old[kRowFlight], ref[kRowFlight], adv[kRowFlight];
                bool in[kRowFlight];
#pragma unroll
                for (int i = 0; i < kRowFlight; i++) {
                    const int r = b0 + i * 32 + lane;
                    const bool live = r < hi;
                    in[i] = live && (p.mask == nullptr || p.mask[r] != 0);
                    if (!kPreference) {
                        now[i] = live ? p.row_loss[r] : 0.0f;
                        old[i] = live ? p.old[r] : 0.0f;
                        ref[i] = live && p.ref ? p.ref[r] : 0.0f;
                        adv[i] = live && !p.by_sequence ? p.advantages[r] : 0.0f;
                    }
                }
                // what the rows' sequences have, before the first store: behind one,
                // each of these loads would wait for the next
                float part[kRowFlight];
#pragma unroll
                for (int i = 0; i < kRowFlight; i++) {
                    const int r0 = b0 + i * 32;
                    part[i] = 0.0f;
                    if (r0 >= hi)
                        continue;
                    const int s = sequence(r0, r0 + lane < hi);
                    in[i] = in[i] && !bad && s >= 0 && (p.offsets == nullptr || s < p.sequences);
                    if (kPreference) {
                        part[i] = in[i] ? __ldcg(p.share + s) : 0.0f;
                    } else if (in[i]) {
                        if (p.by_sequence)
                            adv[i] = p.advantages[s];
                        part[i] = p.reduction == FSDP_POLICY_SEQUENCE ? __ldcg(p.share + s) : 1.0f;
                    }
                }
                float loss_c = 0.0f, kl_c = 0.0f;  // of a few rows
#pragma unroll
                for (int i = 0; i < kRowFlight; i++) {
                    const int r = b0 + i * 32 + lane;
                    float weight = part[i];
                    if (!kPreference && in[i]) {
                        const float k = part[i] * per;
                        const PolicyRow q = policy_row(p, now[i], old[i], ref[i], adv[i], k);
                        weight = q.slope * q.k;
                        loss_c = fmaf(q.term, q.k, loss_c);
                        kl_c += q.kl;
                        clipped += q.cut;
                    }
                    if (r < hi)
                        p.row_weights[r] = weight;
                }
                loss = add(loss, Two{loss_c, 0.0f});
                kl = add(kl, Two{kl_c, 0.0f});
            }
        };
        if (p.offsets) {
            Ends ends(p, lo);
            chunk([&](int r0, bool live) { return ends.at(p, r0, live); });
        } else {
            chunk([](int, bool) { return 0; });
        }
    }
    if (kPreference)
        return;
    loss = block_add(loss, sh2);
    kl = block_add(kl, sh2);
    clipped = block_add(clipped, shi);
    if (threadIdx.x == 0) {
        p.part[block] = loss;
        p.part[blocks + block] = kl;
        p.part_clipped[block] = clipped;
    }
    if (!last_block(p, &last))
        return;
    loss = block_sum(p.part, blocks, sh2);
    kl = block_sum(p.part + blocks, blocks, sh2);
    clipped = block_sum(p.part_clipped, blocks, shi);
    if (threadIdx.x == 0)
        policy_results(p, loss, kl, clipped, counted, bad);
}

// ------------------------------------------------------------- launching ----

constexpr int kWarps = kThreads / 32;
constexpr int kMostBlocks = 1024;
constexpr int kMostChunks = kMostBlocks * kWarps;

// How the rows are cut. The number of multiprocessors is no part of it: the
// workspace is asked for without a device.
void cut(TuneParams &p, const TuneArgs &a)
{
    p.rows = (int)a.rows;
    p.sequences = (int)a.sequences;
    const int64_t want = (a.rows + kMostChunks - 1) / kMostChunks;
    p.chunk = (int)ceil_to(want < 1 ? 1 : want, 32 * kPerThread);
    p.chunks = (int)((a.rows + p.chunk - 1) / p.chunk);
    const int64_t blocks = ((int64_t)p.chunks + kWarps - 1) / kWarps, seq = (a.sequences + kWarps - 1) / kWarps;
    p.blocks = (int)(blocks < 1 ? 1 : blocks);
    p.seq_blocks = (int)(seq < 1 ? 1 : seq < kMostBlocks ? seq : kMostBlocks);
}

void carve(TuneParams &p, void *base, int64_t *bytes)
{
    Carver c(base);
    const int64_t pieces = (int64_t)p.chunks + p.sequences;
    p.done = c.take<int>(1);
    p.bad = c.take<int>(kMostBlocks);
    p.counted = c.take<int>(kMostBlocks);
    p.filled = c.take<int>(kMostBlocks);
    p.part_clipped = c.take<int>(kMostBlocks);
    p.part = c.take<Two>(2 * kMostBlocks);
    p.piece = c.take<Two>(pieces);
    p.piece_count = c.take<int>(pieces);
    p.term = c.take<float>(p.sequences / 2);
    p.share = c.take<float>(p.sequences);
    *bytes = c.used();
}

Two split(double v)
{
    const float hi = (float)v;
    return Two{hi, std::isinf(hi) ? 0.0f : (float)(v - (double)hi)};
}

TuneParams params(const TuneArgs &a, void *workspace)
{
    TuneParams p{};
    cut(p, a);
    int64_t bytes;
    carve(p, workspace, &bytes);
    p.row_loss = a.row_loss, p.ref = a.ref, p.offsets = a.offsets, p.mask = a.mask;
    p.loss = a.loss, p.row_weights = a.row_weights, p.margins = a.margins;
    p.beta = split(a.beta), p.smoothing = (float)a.smoothing, p.average = a.average;
    p.old = a.old, p.advantages = a.advantages, p.by_sequence = a.by_sequence, p.reduction = a.reduction;
    p.low = (float)(1.0 - a.clip_low), p.high = (float)(1.0 + a.clip_high), p.kl_coef = (float)a.kl_coef;
    p.log_low = split(std::log1p(-a.clip_low)), p.log_high = split(std::log1p(a.clip_high));
    p.kl = a.kl, p.clipped = a.clipped;
    return p;
}

bool one_block(const TuneArgs &a) { return a.rows <= kOneBlockRows && a.sequences <= kOneBlockSequences; }

template <bool kPreference>
fsdp_status launch_tune(const TuneArgs &a, void *workspace, bool sums, int dev, cudaStream_t s, const char *what)
{
    const TuneParams p = params(a, workspace);
    if (one_block(a)) {
        constexpr int kSmem = kLists + (kPreference ? (kOneBlockSequences + kOneBlockRows) * 8 : 0);
        if (kSmem > 48 * 1024) {
            static std::atomic<uint64_t> ready{0};  // devices (of the first 64) whose attribute is set
            const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
            if (!(ready.load(std::memory_order_relaxed) & bit)) {
                const cudaError_t e =
                    cudaFuncSetAttribute(small_kernel<kPreference>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
                if (e != cudaSuccess)
                    return set_error(FSDP_ECUDA, "%s: cudaFuncSetAttribute: %s", what, cudaGetErrorString(e));
                ready.fetch_or(bit, std::memory_order_relaxed);
            }
        }
        return launch(what, small_kernel<kPreference>, 1, kOneBlock, kSmem, s, 1, p);
    }
    fsdp_status st = launch(what, count_kernel<kPreference>, (unsigned)p.blocks, kThreads, 0, s, 1, p);
    if (st == FSDP_OK && sums)
        st = launch(what, sum_kernel<kPreference>, (unsigned)p.seq_blocks, kThreads, 0, s, 1, p);
    if (st == FSDP_OK && (p.rows > 0 || !kPreference))
        st = launch(what, row_kernel<kPreference>, (unsigned)p.blocks, kThreads, 0, s, 1, p);
    return st;
}

}  // namespace

int64_t tune_workspace(const TuneArgs &a)
{
    TuneParams p{};
    cut(p, a);
    int64_t bytes;
    carve(p, nullptr, &bytes);
    return one_block(a) ? 0 : bytes;
}

fsdp_status launch_preference_loss(const TuneArgs &a, void *workspace, int dev, void *stream)
{
    return launch_tune<true>(a, workspace, true, dev, static_cast<cudaStream_t>(stream), "preference_loss");
}

fsdp_status launch_policy_loss(const TuneArgs &a, void *workspace, int dev, void *stream)
{
    return launch_tune<false>(a, workspace, a.reduction == FSDP_POLICY_SEQUENCE, dev, static_cast<cudaStream_t>(stream),
                              "policy_loss");
}

}  // namespace fsdp
