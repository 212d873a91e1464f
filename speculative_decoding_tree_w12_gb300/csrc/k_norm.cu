// Norms around a block (sm_103a).
//
//  * k_gdn_norm: a recurrent layer's outputs, head by head, as the next linear
//    reads them.  With rms(x) = x / sqrt(mean(x^2) + eps) over a head's 128
//    values and gate = z / (1 + exp(-z)):
//        x = rms(o) w gate      or, with the gate first,      x = rms(o gate) w
//  * k_block_norm: between two blocks,
//        h' = h + scale t,  t = y or rms(y) w_post over a row,
//        x  = rms(h') w_pre.
//
// Both are bound by memory: one pass, each input read once and each output
// written once, sums in FP32 in registers.  x is taken from the FP32 h', not
// from the value that is stored: one rounding less in every layer.
//
// 16384 rows of 32 heads with their gate (537 MB): 74.9 us, 7.2 TB/s.  Between two blocks of 5120 values, 16384 rows: 98.9 us BF16
// (6.8 TB/s), 148.4 us FP32 with a norm behind the block (6.8); 192 rows 2.4 and 3.8 us, call after call.  (76.7, 99.8, 149.6, 2.75
// and 4.2 if a launch waits for the one before it to end before it begins.)
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "w12_device.cuh"
#include "w12_internal.h"

namespace {

constexpr int kHead = 128;

__device__ __forceinline__ float lo16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi16(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

__device__ __forceinline__ void unpack8(const uint4 &w, float (&x)[8])
{
    x[0] = lo16(w.x);
    x[1] = hi16(w.x);
    x[2] = lo16(w.y);
    x[3] = hi16(w.y);
    x[4] = lo16(w.z);
    x[5] = hi16(w.z);
    x[6] = lo16(w.w);
    x[7] = hi16(w.w);
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    uint32_t d;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8])
{
    return make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7]));
}

// z / (1 + exp(-z)), for z < 0 as z exp(z) / (1 + exp(z)): 1 + exp(-z) leaves FP32's range at z = -88.7.  exp(-|z|) is held 2^32 times
// as large until the last product, so that it has all its bits where the result has.  Off by (8 + 0.45 |z|) 2^-23 at most: 2^x by 2
// units, the reciprocal by 1, log2(e) by 0.12 |z|, the exponent by half its last place (4 units up to 16, 22 up to 128), products by 2.
// That is 2^-17 of a result where the gate closes, in front of a rounding of 2^-9.  (16384 rows of 32 heads 74.9 us; 78.5 with the gate behind
// the norm and 82.4 in front of it with an exponential that is right to a bit or two.)
__device__ __forceinline__ float silu(float z)
{
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(fmaf(fabsf(z), -1.44269504f, 32.f)));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(fmaf(e, 0x1p-32f, 1.f)));
    return z < 0.f ? (z * e) * (r * 0x1p-32f) : z * r;
}

// ---------------------------------------------------------------------------
// outputs of a recurrent layer
// ---------------------------------------------------------------------------
//
// Sixteen lanes to a head (eight values each: 32 bytes of o, 16 of z and of
// x), so a warp takes two heads at a time and its sum needs four shuffles.

constexpr int kNormThreads = 256;

struct GdnNormParams {
    const float *o;
    const uint16_t *z, *w;
    uint16_t *x;
    int64_t z_stride, x_stride;
    uint32_t H, items;      // items = rows * heads
    float eps;
};

template <bool kGate, bool kFirst>
__global__ void __launch_bounds__(kNormThreads) k_gdn_norm(const GdnNormParams p)
{
    w12d::pdl_wait();
    w12d::pdl_launch_dependents();
    const uint32_t item = blockIdx.x * (uint32_t)(kNormThreads / 16) + (threadIdx.x >> 4);
    const int c = (threadIdx.x & 15) * 8;
    const bool live = item < p.items;      // (the other half of the warp takes part in the shuffles)
    const uint32_t row = live ? item / p.H : 0, head = live ? item - row * p.H : 0;
    float x[8], g[8], w[8];
    {
        const float4 *src = reinterpret_cast<const float4 *>(p.o + (size_t)(live ? item : 0) * kHead + c);
        const float4 a = src[0], b = src[1];
        x[0] = a.x;
        x[1] = a.y;
        x[2] = a.z;
        x[3] = a.w;
        x[4] = b.x;
        x[5] = b.y;
        x[6] = b.z;
        x[7] = b.w;
    }
    if (kGate) unpack8(*reinterpret_cast<const uint4 *>(p.z + row * p.z_stride + head * kHead + c), g);
    unpack8(*reinterpret_cast<const uint4 *>(p.w + c), w);
    if (kGate) {
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] = silu(g[i]);
    }
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (kGate && kFirst) x[i] *= g[i];
        sum = fmaf(x[i], x[i], sum);
    }
#pragma unroll
    for (int s = 8; s; s >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
    const float r = rsqrtf(fmaf(sum, 1.f / kHead, p.eps));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        x[i] *= r * w[i];
        if (kGate && !kFirst) x[i] *= g[i];
    }
    if (live) *reinterpret_cast<uint4 *>(p.x + row * p.x_stride + head * kHead + c) = pack8(x);
}

// ---------------------------------------------------------------------------
// between two blocks
// ---------------------------------------------------------------------------
//
// One CTA to a row, kV pieces of eight values to a thread, kept in registers
// between the sums.  Every thread reads its pieces before its first barrier
// and writes the same places after it, so h' may be h and x may be y.

struct BlockNormParams {
    const void *h;
    void *h_out;
    const uint16_t *y, *post, *pre;
    uint16_t *x;
    int64_t h_stride, ho_stride, y_stride, x_stride;
    int32_t pieces;         // n / 8
    float scale, eps, inv_n;
};

__device__ __forceinline__ float row_sum(float v, float *part, int warps)
{
#pragma unroll
    for (int s = 16; s; s >>= 1) v += __shfl_xor_sync(0xffffffffu, v, s);
    const int lane = threadIdx.x & 31;
    if (lane == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    float t = lane < warps ? part[lane] : 0.f;
#pragma unroll
    for (int s = 16; s; s >>= 1) t += __shfl_xor_sync(0xffffffffu, t, s);
    return t;
}

template <bool kF32, int kV>
__global__ void __launch_bounds__(1024) k_block_norm(const BlockNormParams p)
{
    w12d::pdl_wait();
    w12d::pdl_launch_dependents();
    __shared__ float part[2][32];
    const size_t row = blockIdx.x;
    const int warps = blockDim.x >> 5;
    float h[kV][8], y[kV][8];
    float sum = 0.f;
#pragma unroll
    for (int v = 0; v < kV; ++v) {
        const int i = threadIdx.x + v * blockDim.x;
#pragma unroll
        for (int e = 0; e < 8; ++e) h[v][e] = y[v][e] = 0.f;
        if (i >= p.pieces) continue;
        if (kF32) {
            const float4 *src = reinterpret_cast<const float4 *>(static_cast<const float *>(p.h) + row * p.h_stride) + 2 * i;
            const float4 a = src[0], b = src[1];
            h[v][0] = a.x;
            h[v][1] = a.y;
            h[v][2] = a.z;
            h[v][3] = a.w;
            h[v][4] = b.x;
            h[v][5] = b.y;
            h[v][6] = b.z;
            h[v][7] = b.w;
        } else {
            unpack8(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.h) + row * p.h_stride)[i], h[v]);
        }
        if (p.y) unpack8(reinterpret_cast<const uint4 *>(p.y + row * p.y_stride)[i], y[v]);
    }
    if (p.post) {
#pragma unroll
        for (int v = 0; v < kV; ++v)
#pragma unroll
            for (int e = 0; e < 8; ++e) sum = fmaf(y[v][e], y[v][e], sum);
        const float r = rsqrtf(fmaf(row_sum(sum, part[0], warps), p.inv_n, p.eps));
#pragma unroll
        for (int v = 0; v < kV; ++v) {
            const int i = threadIdx.x + v * blockDim.x;
            if (i >= p.pieces) continue;
            float w[8];
            unpack8(reinterpret_cast<const uint4 *>(p.post)[i], w);
#pragma unroll
            for (int e = 0; e < 8; ++e) y[v][e] *= r * w[e];
        }
    }
    if (p.y) {
#pragma unroll
        for (int v = 0; v < kV; ++v) {
            const int i = threadIdx.x + v * blockDim.x;
#pragma unroll
            for (int e = 0; e < 8; ++e) h[v][e] = fmaf(p.scale, y[v][e], h[v][e]);
            if (i >= p.pieces) continue;
            if (kF32) {
                float4 *dst = reinterpret_cast<float4 *>(static_cast<float *>(p.h_out) + row * p.ho_stride) + 2 * i;
                dst[0] = make_float4(h[v][0], h[v][1], h[v][2], h[v][3]);
                dst[1] = make_float4(h[v][4], h[v][5], h[v][6], h[v][7]);
            } else {
                reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.h_out) + row * p.ho_stride)[i] = pack8(h[v]);
            }
        }
    }
    if (!p.pre) return;
    sum = 0.f;
#pragma unroll
    for (int v = 0; v < kV; ++v)
#pragma unroll
        for (int e = 0; e < 8; ++e) sum = fmaf(h[v][e], h[v][e], sum);
    const float r = rsqrtf(fmaf(row_sum(sum, part[1], warps), p.inv_n, p.eps));
#pragma unroll
    for (int v = 0; v < kV; ++v) {
        const int i = threadIdx.x + v * blockDim.x;
        if (i >= p.pieces) continue;
        float w[8];
        unpack8(reinterpret_cast<const uint4 *>(p.pre)[i], w);
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] *= h[v][e] * r;
        reinterpret_cast<uint4 *>(p.x + row * p.x_stride)[i] = pack8(w);
    }
}

template <class P>
int launch(void (*kern)(P), uint32_t grid, int threads, const P &p, void *stream)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute behind{};                 // begins while the launch before it ends, and waits for that first of all
    behind.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    behind.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &behind;
    cfg.numAttrs = 1;
    return (int)cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace

namespace w12i {

int launch_gdn_norm(const GdnNormArgs &a, void *stream)
{
    GdnNormParams p{};
    p.o = a.o;
    p.z = a.z;
    p.w = a.w;
    p.x = a.x;
    p.z_stride = a.z_stride;
    p.x_stride = a.x_stride;
    p.H = (uint32_t)a.H;
    p.items = (uint32_t)a.H * (uint32_t)a.rows;
    p.eps = a.eps;
    const uint32_t per = kNormThreads / 16, grid = p.items / per + (p.items % per != 0);
    const auto kern = !p.z ? k_gdn_norm<false, false> : a.gate_first ? k_gdn_norm<true, true> : k_gdn_norm<true, false>;
    return launch(kern, grid, kNormThreads, p, stream);
}

int launch_block_norm(const BlockNormArgs &a, void *stream)
{
    BlockNormParams p{};
    p.h = a.h;
    p.h_out = a.h_out;
    p.y = a.y;
    p.post = a.post;
    p.pre = a.pre;
    p.x = a.x;
    p.h_stride = a.h_stride;
    p.ho_stride = a.ho_stride;
    p.y_stride = a.y_stride;
    p.x_stride = a.x_stride;
    p.pieces = (int32_t)(a.n / 8);
    p.scale = a.scale;
    p.eps = a.eps;
    p.inv_n = 1.f / (float)a.n;
    // As many threads as leave one piece to each, two beyond 1024 threads.  (16384 BF16 rows of 5120 values, without overlap: one
    // piece 99.8 us, two 115.0; of 2560: 49.1 and 54.9; 192 rows of 8192: 3.5 and 3.3.  Rows of 16384, which only go with two: 391 us,
    // 5.5 TB/s.)
    const int v = p.pieces <= 1024 ? 1 : 2;
    const int threads = ((p.pieces + v - 1) / v + 31) / 32 * 32;
    const auto k16 = v == 1 ? k_block_norm<false, 1> : k_block_norm<false, 2>;
    const auto k32 = v == 1 ? k_block_norm<true, 1> : k_block_norm<true, 2>;
    return launch(a.h_f32 ? k32 : k16, (uint32_t)a.rows, threads, p, stream);
}

}  // namespace w12i
