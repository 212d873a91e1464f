// Recurrent (Gated DeltaNet) layer: one new token of every request (sm_103a).
//
// With gate a, strength b, key k, value v, query q and the state S (d_v x d_k)
//     u = b (v - a S k),   S' = a S + u k^T,   o = S' q = a S q + u (k.q),
// so one pass over S gives both products (S k and S q), the new state and the
// output.  Bound by memory: 128 KB of state in and out to 1.3 KB of rows.
//
// Eight lanes share a row of S (sixteen of its columns each, as four float4
// eight lanes apart), so a load of a warp covers four rows by whole 128-byte
// lines and each sum takes three shuffles; a warp takes eight rows, every load
// of which is asked for before the first is used.  Four CTAs of 32 rows to a
// head: one request of 32 heads puts 128 CTAs on the machine.
//
// 256 requests of 32 heads (1.08 GB), call after call: 172.6 us, 6.3 TB/s; 24 requests 17.1 us, 5.9 TB/s (18.8 if a launch waits for
// the one before it to end before it begins); one request 4.1 us by itself, which is the launch and one way to memory and back.
#include <cuda_runtime.h>

#include "w12_device.cuh"
#include "w12_internal.h"

namespace {

constexpr int kD = 128;
constexpr int kStepThreads = 128;
constexpr int kStepRows = 32;      // of the state, a CTA

struct GdnStepParams {
    const float *S0;               // may be null: zero
    float *state, *o;
    const uint16_t *q, *k, *v;
    const float *alpha, *beta;
    int64_t q_stride, k_stride, v_stride;
    int32_t H, group;              // group: value heads of a key head
};

__device__ __forceinline__ float bf(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }

__device__ __forceinline__ float4 bf4(const uint16_t *p)
{
    const uint2 w = *reinterpret_cast<const uint2 *>(p);
    return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                       __uint_as_float(w.y & 0xffff0000u));
}

__device__ __forceinline__ float dot4(const float4 &a, const float4 &b, float c)
{
    return fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, c))));
}

__device__ __forceinline__ float sum8(float x)
{
#pragma unroll
    for (int s = 4; s; s >>= 1) x += __shfl_xor_sync(0xffffffffu, x, s);
    return x;
}

__global__ void __launch_bounds__(kStepThreads) k_gdn_step(const GdnStepParams p)
{
    w12d::pdl_wait();
    w12d::pdl_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c0 = (lane & 7) * 4, h = blockIdx.y;
    const size_t r = blockIdx.x;
    const int row = blockIdx.z * kStepRows + warp * 8 + (lane >> 3);      // and row + 4
    const size_t at = ((r * p.H + h) * kD + row) * kD + c0;
    float4 s[2][4], kk[4], qq[4];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            s[i][e] = p.S0 ? *reinterpret_cast<const float4 *>(p.S0 + at + i * 4 * kD + e * 32) : make_float4(0.f, 0.f, 0.f, 0.f);
    const uint16_t *kp = p.k + r * p.k_stride + (h / p.group) * kD + c0;
    const uint16_t *qp = p.q + r * p.q_stride + (h / p.group) * kD + c0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        kk[e] = bf4(kp + e * 32);
        qq[e] = bf4(qp + e * 32);
    }
    const float a = p.alpha[r * p.H + h], b = p.beta[r * p.H + h];
    float vv[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) vv[i] = bf(p.v[r * p.v_stride + h * kD + row + 4 * i]);
    float kq = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) kq = dot4(kk[e], qq[e], kq);
    kq = sum8(kq);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        float sk = 0.f, sq = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            sk = dot4(s[i][e], kk[e], sk);
            sq = dot4(s[i][e], qq[e], sq);
        }
        sk = sum8(sk);
        sq = sum8(sq);
        const float u = b * (vv[i] - a * sk);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float4 &x = s[i][e];
            *reinterpret_cast<float4 *>(p.state + at + i * 4 * kD + e * 32) =
                make_float4(fmaf(u, kk[e].x, a * x.x), fmaf(u, kk[e].y, a * x.y), fmaf(u, kk[e].z, a * x.z),
                            fmaf(u, kk[e].w, a * x.w));
        }
        if ((lane & 7) == 0) p.o[(r * p.H + h) * kD + row + 4 * i] = fmaf(u, kq, a * sq);
    }
}

}  // namespace

namespace w12i {

int launch_gdn_step(const GdnSeqArgs &a, void *stream)
{
    GdnStepParams p{};
    p.S0 = a.S0;
    p.state = a.state;
    p.o = a.o;
    p.q = a.q;
    p.k = a.k;
    p.v = a.v;
    p.alpha = a.alpha;
    p.beta = a.beta;
    p.q_stride = a.q_stride;
    p.k_stride = a.k_stride;
    p.v_stride = a.v_stride;
    p.H = a.H;
    p.group = a.H / a.Hk;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(a.n_req, a.H, kD / kStepRows);
    cfg.blockDim = dim3(kStepThreads);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute behind{};                 // begins while the launch before it ends, and waits for that first of all
    behind.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    behind.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &behind;
    cfg.numAttrs = 1;
    return (int)cudaLaunchKernelEx(&cfg, k_gdn_step, p);
}

}  // namespace w12i
