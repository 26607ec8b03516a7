// fsdp_dropout.cu -- dropout whose mask is never stored, for sm_103a:
//
//   y = residual + (draw < keep_of ? x * 65536 / keep_of : 0)
//
// The draws are the 16-bit halves of Philox4x32-10 (Salmon, Moraes, Dror,
// Shaw: Parallel random numbers, as easy as 1, 2, 3; 2011), eight to a counter
// (column / 8, row, offset) under the key `seed`: any element's mask follows
// from its place alone, so the backward pass makes it again, whatever strides,
// alignment or grid the two have.
//
// Bound by HBM, 16384 x 4096: bf16 with a residual 61.0 us, 6.6 TB/s (0.97 of a
// plain copy's rate), fp32 115.4 with and 78.2 us without, 6.9 TB/s; bf16 alone
// 49.4 us, 5.4 TB/s, by issue slots: ten rounds of two wide multiplications per
// 8 elements. With draws of 32 bits, and so per 4, bf16 takes 72.0 and 68.4 us.
// Rows that start anywhere: 16384 x 4095 fp32 84 us, bf16 79 (two bytes a lane:
// issue slots are 70 % active, DRAM a third).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "fsdp_divide.cuh"
#include "fsdp_launch.cuh"

namespace fsdp {
namespace {

constexpr int kThreads = 256;

struct DropoutParams {
    int64_t ldx, ldr, ldy;
    int64_t total;  // groups of 8 columns
    Divide groups;  // of a row
    int cols;
    const void *x, *residual;
    void *y;
    float scale;
    uint32_t last;  // keep_of * 65536 - 1
    bool none;      // keep_of = 0
    int units;      // of a row: kUnit columns each (kRows)
    uint64_t seed, offset;
    const int64_t *offset_more;
};

__device__ __forceinline__ void philox(uint32_t (&c)[4], uint32_t k0, uint32_t k1)
{
#pragma unroll
    for (int i = 0; i < 10; i++) {
        const uint64_t a = (uint64_t)c[0] * 0xD2511F53u, b = (uint64_t)c[2] * 0xCD9E8D57u;
        c[0] = (uint32_t)(b >> 32) ^ c[1] ^ k0;
        c[2] = (uint32_t)(a >> 32) ^ c[3] ^ k1;
        c[1] = (uint32_t)b;
        c[3] = (uint32_t)a;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
}

// Element i of a group stays: its half of word i / 2 is below keep_of. `last`
// is keep_of * 65536 - 1: the high half needs no shift to be compared, and
// keep_of = 65536 no case of its own (keep_of = 0 has one).
__device__ __forceinline__ bool stays(const uint32_t (&c)[4], int i, uint32_t last)
{
    return (i % 2 ? c[i / 2] : c[i / 2] << 16) <= last;
}
__device__ __forceinline__ void draw(const DropoutParams &p, uint32_t row, uint32_t group, uint64_t offset, uint32_t (&c)[4])
{
    c[0] = group;
    c[1] = row;
    c[2] = (uint32_t)offset;
    c[3] = (uint32_t)(offset >> 32);
    philox(c, (uint32_t)p.seed, (uint32_t)(p.seed >> 32));
}
// Which of a group's 8 elements stay, a bit each.
__device__ __forceinline__ uint32_t kept(const DropoutParams &p, uint32_t row, uint32_t group, uint64_t offset)
{
    uint32_t c[4], bits = 0;
    draw(p, row, group, offset, c);
#pragma unroll
    for (int i = 0; i < 8; i++)
        bits |= (stays(c, i, p.last) ? 1u : 0u) << i;
    return p.none ? 0 : bits;
}

__device__ __forceinline__ float load1(const uint16_t *p) { return __uint_as_float((uint32_t)*p << 16); }
__device__ __forceinline__ float load1(const float *p) { return *p; }
__device__ __forceinline__ void store1(uint16_t *p, float v) { *p = __bfloat16_as_ushort(__float2bfloat16_rn(v)); }
__device__ __forceinline__ void store1(float *p, float v) { *p = v; }

// Eight elements as they lie, 16 bytes a piece.
template <typename T>
struct Eight {
    static constexpr int kPieces = (int)sizeof(T) / 2;
    uint4 raw[kPieces];
    __device__ __forceinline__ void load(const T *p)
    {
#pragma unroll
        for (int i = 0; i < kPieces; i++)
            asm volatile("ld.global.L1::no_allocate.v4.b32 {%0,%1,%2,%3}, [%4];"
                         : "=r"(raw[i].x), "=r"(raw[i].y), "=r"(raw[i].z), "=r"(raw[i].w)
                         : "l"(p + i * (8 / kPieces)));
    }
    __device__ __forceinline__ void store(T *p) const
    {
#pragma unroll
        for (int i = 0; i < kPieces; i++)
            *reinterpret_cast<uint4 *>(p + i * (8 / kPieces)) = raw[i];
    }
    __device__ __forceinline__ float get(int i) const { return load1(reinterpret_cast<const T *>(raw) + i); }
    __device__ __forceinline__ void set(int i, float v) { store1(reinterpret_cast<T *>(raw) + i, v); }
};

__device__ __forceinline__ void place(const DropoutParams &p, int64_t g, int64_t &row, int &group)
{
    if (p.total < (int64_t)1 << 31) {
        const uint32_t r = p.groups((uint32_t)g);
        row = r;
        group = (int)((uint32_t)g - r * (uint32_t)p.groups.d);
    } else {
        row = g / p.groups.d;
        group = (int)(g - row * p.groups.d);
    }
}

// How the elements are dealt out.
//   kVector   a thread per group: rows are whole groups and start on 16 bytes
//   kRows     a warp per 256 columns of a row, lanes side by side on elements;
//             an element's bit comes from the lane that has made its group's
//   kAny      the same for a warp's 32 groups, wherever their rows are: narrow
//             rows, which would leave most of the 256 columns empty
enum Deal { kVector, kRows, kAny };
constexpr int kUnit = 256;

template <typename T, int kDeal, bool kResidual>
__global__ void __launch_bounds__(kThreads) dropout_kernel(const DropoutParams p)
{
    launch_wait();
    launch_next();
    const T *x = static_cast<const T *>(p.x), *res = static_cast<const T *>(p.residual);
    T *y = static_cast<T *>(p.y);
    const uint64_t offset = p.offset + (p.offset_more ? (uint64_t)*p.offset_more : 0);
    const int64_t step = (int64_t)gridDim.x * kThreads;
    const int lane = threadIdx.x % 32;
    int64_t g = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if constexpr (kDeal == kVector) {
        for (; g < p.total; g += step) {
            Eight<T> a, b;
            int64_t row;
            int group;
            place(p, g, row, group);
            a.load(x + row * p.ldx + group * 8);
            if (kResidual)
                b.load(res + row * p.ldr + group * 8);
            uint32_t c[4];
            draw(p, (uint32_t)row, (uint32_t)group, offset, c);
#pragma unroll
            for (int i = 0; i < 8; i++) {
                const float r = kResidual ? b.get(i) : 0.0f;
                a.set(i, stays(c, i, p.last) && !p.none ? fmaf(a.get(i), p.scale, r) : r);
            }
            a.store(y + row * p.ldy + group * 8);
        }
    } else if constexpr (kDeal == kRows) {
        // p.total: units
        for (int64_t u = g / 32; u < p.total; u += step / 32) {
            const int64_t row = u / p.units;
            const int col0 = (int)(u - row * p.units) * kUnit, left = p.cols - col0 - lane;
            const T *from = x + row * p.ldx + col0 + lane, *add = res + row * p.ldr + col0 + lane;
            T *to = y + row * p.ldy + col0 + lane;
            float v[8], r[8];
#pragma unroll
            for (int j = 0; j < 8; j++) {
                v[j] = j * 32 < left ? load1(from + j * 32) : 0.0f;
                r[j] = kResidual && j * 32 < left ? load1(add + j * 32) : 0.0f;
            }
            const uint32_t bits = kept(p, (uint32_t)row, (uint32_t)(col0 / 8 + lane), offset);
#pragma unroll
            for (int j = 0; j < 8; j++) {
                const uint32_t m = __shfl_sync(0xffffffffu, bits, j * 4 + lane / 8);
                if (j * 32 < left)
                    store1(to + j * 32, m >> (lane % 8) & 1 ? fmaf(v[j], p.scale, r[j]) : r[j]);
            }
        }
    } else {
        // whole warps: the last one's lanes past the end take part without a group
        for (g -= lane; g < p.total; g += step) {
            const int64_t mine = g + lane;
            int64_t row = 0;
            int group = 0;
            uint32_t bits = 0;
            if (mine < p.total) {
                place(p, mine, row, group);
                bits = kept(p, (uint32_t)row, (uint32_t)group, offset);
            }
            float v[8], r[8];
            int64_t at[8];
            int col[8];
            bool live[8];
#pragma unroll
            for (int j = 0; j < 8; j++) {
                const int from = j * 4 + lane / 8;
                at[j] = __shfl_sync(0xffffffffu, row, from);
                col[j] = __shfl_sync(0xffffffffu, group, from) * 8 + lane % 8;
                live[j] = g + from < p.total && col[j] < p.cols;
                v[j] = live[j] ? load1(x + at[j] * p.ldx + col[j]) : 0.0f;
                r[j] = kResidual && live[j] ? load1(res + at[j] * p.ldr + col[j]) : 0.0f;
            }
#pragma unroll
            for (int j = 0; j < 8; j++) {
                const uint32_t m = __shfl_sync(0xffffffffu, bits, j * 4 + lane / 8);
                if (live[j])
                    store1(y + at[j] * p.ldy + col[j], m >> (lane % 8) & 1 ? fmaf(v[j], p.scale, r[j]) : r[j]);
            }
        }
    }
}

// Rows from here on are dealt out by units: fp32 of 101 columns 108 us against
// 131, of 259 109 against 164; of 57 columns 132 against 102 (40 to 50 million
// elements each).
constexpr int kRowsCols = 96;

template <typename T, int kDeal>
fsdp_status launch_dealt(const DropoutArgs &a, const DropoutParams &p, int64_t threads, int64_t most, cudaStream_t stream)
{
    const int64_t blocks = (threads + kThreads - 1) / kThreads;
    const dim3 grid((unsigned)(blocks < most ? blocks : most));
    return a.residual ? launch("dropout", dropout_kernel<T, kDeal, true>, grid, kThreads, 0, stream, 1, p)
                      : launch("dropout", dropout_kernel<T, kDeal, false>, grid, kThreads, 0, stream, 1, p);
}

template <typename T>
fsdp_status launch_as(const DropoutArgs &a, DropoutParams p, int dev, cudaStream_t stream)
{
    auto on_16 = [](const void *q, int64_t ld) {
        return ((reinterpret_cast<uintptr_t>(q) | (uintptr_t)(ld * (int64_t)sizeof(T))) & 15u) == 0;
    };
    const int64_t sms = device_sms(dev);
    // bf16, which is the closer to issue slots, gains from threads that go on to
    // a next group (16384 x 4096: 49.4 us, with a group a thread 58.7; with a
    // residual 61.1 and 61.0); fp32 from blocks that are replaced (83.1 and 78.2)
    if (a.cols % 8 == 0 && on_16(a.x, a.ldx) && on_16(a.y, a.ldy) && (a.residual == nullptr || on_16(a.residual, a.ldr)))
        return launch_dealt<T, kVector>(a, p, p.total, sizeof(T) == 2 ? 32 * sms : 1 << 30, stream);
    if (a.cols >= kRowsCols) {
        p.total = a.rows * p.units;
        return launch_dealt<T, kRows>(a, p, p.total * 32, 32 * sms, stream);
    }
    return launch_dealt<T, kAny>(a, p, p.total, 32 * sms, stream);
}

}  // namespace

fsdp_status launch_dropout(const DropoutArgs &a, int dev, void *stream)
{
    const int64_t groups = (a.cols + 7) / 8;
    DropoutParams p{a.ldx, a.ldr, a.ldy, a.rows * groups, Divide((int)groups), (int)a.cols, a.x, a.residual, a.y,
                    a.keep_of ? 65536.0f / (float)a.keep_of : 0.0f, a.keep_of * 65536u - 1u, a.keep_of == 0,
                    (int)((a.cols + kUnit - 1) / kUnit), a.seed, a.offset, a.offset_more};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return a.dtype == FSDP_BF16 ? launch_as<uint16_t>(a, p, dev, s) : launch_as<float>(a, p, dev, s);
}

}  // namespace fsdp
