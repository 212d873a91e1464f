// Attention of a draft tree's rows over a paged 8-bit KV cache and over the
// rows' own root paths.
//
// Mathematics.  Row i of request r stands at position len_r + depth_i.  Its
// output is softmax over the len_r cached tokens and over i's ancestors and i
// itself: every row of a request sees the whole cached context, so that part
// has no mask but its end; the tree part runs over the root path alone (at
// most kMaxDepth + 1 rows), so it needs no mask either, and whatever stands in
// a row off the path cannot reach the output.
//
// The cached part is split over the tokens; each part leaves its FP32 sums
// with their maximum and normaliser, and the join kernel merges them with the
// root path's.
#include <cuda_runtime.h>

#include <cstdint>

#include "w12_device.cuh"
#include "w12_kv.cuh"

namespace {

using namespace w12d;
using namespace w12i;

constexpr int kD = kKvDim;
constexpr int kPath = kMaxDepth + 1;       // rows of a root path
constexpr float kLog2e = 1.4426950408889634f;

struct AttnParams {
    int32_t H, Hq, G, bt, n_blocks, max_blocks, n_req, R, S;
    int64_t q_stride, k_stride, v_stride;
    const uint8_t *kc, *vc;
    const float *ks, *vs;
    const int32_t *table, *len, *off, *parent, *req;
    const uint8_t *depth;
    const uint16_t *q, *k, *v;
    RopeArgs rope;
    float scale2;                           // softmax scale * log2(e)
    uint16_t *out;
    float *part;                            // [R * Hq][S][kD + 2]
    int32_t *status;
};

__device__ __forceinline__ void fail(int32_t *status) { atomicCAS(status, 0, (int32_t)W12_E_INVAL); }

// the request of a row, or -1 where the tree's arrays contradict each other or the cache
__device__ __forceinline__ int request_of(const AttnParams &p, int row)
{
    const int r = p.req[row];
    if (r < 0 || r >= p.n_req) return -1;
    const int lo = p.off[r], hi = p.off[r + 1], n = p.len[r];
    if (lo < 0 || hi > p.R || row < lo || row >= hi) return -1;
    if (n < 0 || (int64_t)n > (int64_t)p.max_blocks * p.bt) return -1;
    if (p.rope.rot && n + (int)p.depth[row] >= p.rope.max_pos) return -1;
    return r;
}

__global__ void __launch_bounds__(128) k_attn_part(const AttnParams p)
{
    __shared__ float sq[kD], sp[128], red[8];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int row = blockIdx.x / p.Hq, hq = blockIdx.x % p.Hq, h = hq / p.G;
    const int r = request_of(p, row);
    float *out = p.part + ((int64_t)blockIdx.x * p.S + blockIdx.y) * (kD + 2);
    const int n = r < 0 ? 0 : p.len[r];
    const int per = ((n + p.S - 1) / p.S + 127) / 128 * 128;
    const int t0 = blockIdx.y * per, t1 = min(n, t0 + per);
    float m = -INFINITY, l = 0.f, o = 0.f;
    if (t0 < t1) {
        sq[tid] = rotated(p.q + row * p.q_stride + hq * kD, tid, n + p.depth[row], p.rope) * p.scale2;
        __syncthreads();
        for (int t = t0; t < t1; t += 128) {
            const int tok = t + tid;
            float s = -INFINITY;
            if (tok < t1) {
                const int b = p.table[(int64_t)r * p.max_blocks + tok / p.bt];
                if (b < 0 || b >= p.n_blocks) fail(p.status);
                else {
                    const int64_t bh = (int64_t)b * p.H + h;
                    const uint8_t *kr = p.kc + (bh * p.bt + tok % p.bt) * kD;
                    s = 0.f;
                    for (int d = 0; d < kD; ++d) s += sq[d] * e4m3_f32(kr[d]);
                    s *= p.ks[bh];
                }
            }
            float tm = s;
            for (int d = 16; d; d >>= 1) tm = fmaxf(tm, __shfl_xor_sync(0xffffffffu, tm, d));
            if (lane == 0) red[warp] = tm;
            __syncthreads();
            tm = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
            const float m1 = fmaxf(m, tm);
            const float base = m1 == -INFINITY ? 0.f : m1;
            const float e = exp2f(s - base), c = exp2f(m - base);
            sp[tid] = e;
            float ts = e;
            for (int d = 16; d; d >>= 1) ts += __shfl_xor_sync(0xffffffffu, ts, d);
            if (lane == 0) red[4 + warp] = ts;
            __syncthreads();
            l = l * c + (red[4] + red[5] + red[6] + red[7]);
            o *= c;
            m = m1;
            for (int i = 0; i < 128 && t + i < t1; ++i) {
                const int b = p.table[(int64_t)r * p.max_blocks + (t + i) / p.bt];
                if (b < 0 || b >= p.n_blocks) continue;
                const int64_t bh = (int64_t)b * p.H + h;
                o += sp[i] * e4m3_f32(p.vc[(bh * kD + tid) * p.bt + (t + i) % p.bt]) * p.vs[bh];
            }
            __syncthreads();
        }
    }
    out[tid] = o;
    if (tid == 0) out[kD] = m, out[kD + 1] = l;
}

// One CTA per row and key/value head: the root path's attention for the G
// query heads of the group, merged with the parts of the cached context.
__global__ void __launch_bounds__(128) k_attn_join(const AttnParams p)
{
    extern __shared__ float sm[];
    float *sk = sm;                                     // [kPath][kD + 1] keys of the path, turned
    float *sv = sk + kPath * (kD + 1);                  // [kPath][kD]
    float *sq = sv + kPath * kD;                        // [G][kD]
    float *ss = sq + p.G * kD;                          // [G][kPath] scores, then weights
    __shared__ int32_t s_parent[kMaxBudget], s_path[kPath + 1], s_n;
    const int tid = threadIdx.x;
    const int row = blockIdx.x, h = blockIdx.y, G = p.G;
    const int r = request_of(p, row);
    const int lo = r < 0 ? row : p.off[r];
    for (int j = lo + tid; j <= row; j += 128) s_parent[j - lo] = p.parent[j];
    __syncthreads();
    if (tid == 0) {
        int n = 0, j = row;
        while (r >= 0 && j >= lo && n <= kPath) {
            s_path[n++] = j;
            const int q = s_parent[j - lo];
            if (q >= j || (p.rope.rot && p.len[r] + (int)p.depth[j] >= p.rope.max_pos)) n = kPath + 1;                  // a parent after its child, a position off the table
            else j = q;
        }
        if (r < 0 || n > kPath || j >= 0) {             // ... or outside the request
            n = 0;
            fail(p.status);
        }
        s_n = n;
    }
    __syncthreads();
    const int nA = s_n;
    uint16_t *o = p.out + ((int64_t)row * p.Hq + h * G) * kD;
    if (nA == 0) {                                      // malformed: zeros, and the status word says so
        for (int i = tid; i < G * kD; i += 128) o[i] = 0;
        return;
    }
    const int n = p.len[r];
    for (int a = 0; a < nA; ++a) {
        const int64_t j = s_path[a];
        sk[a * (kD + 1) + tid] = rotated(p.k + j * p.k_stride + h * kD, tid, n + p.depth[j], p.rope);
        sv[a * kD + tid] = bf16_f32(p.v[j * p.v_stride + h * kD + tid]);
    }
    for (int g = 0; g < G; ++g)
        sq[g * kD + tid] = rotated(p.q + row * p.q_stride + (h * G + g) * kD, tid, n + p.depth[row], p.rope) * p.scale2;
    __syncthreads();
    for (int i = tid; i < G * nA; i += 128) {
        const int g = i / nA, a = i % nA;
        float s = 0.f;
        for (int d = 0; d < kD; ++d) s += sq[g * kD + d] * sk[a * (kD + 1) + d];
        ss[g * kPath + a] = s;
    }
    __syncthreads();
    for (int g = 0; g < G; ++g) {
        const float *part = p.part + ((int64_t)row * p.Hq + h * G + g) * p.S * (kD + 2);
        float m = -INFINITY;
        for (int a = 0; a < nA; ++a) m = fmaxf(m, ss[g * kPath + a]);
        for (int s = 0; s < p.S; ++s) m = fmaxf(m, part[s * (kD + 2) + kD]);
        const float base = m == -INFINITY ? 0.f : m;
        float l = 0.f, x = 0.f;
        for (int a = 0; a < nA; ++a) {
            const float e = exp2f(ss[g * kPath + a] - base);
            l += e;
            x += e * sv[a * kD + tid];
        }
        for (int s = 0; s < p.S; ++s) {
            const float *q = part + s * (kD + 2);
            const float c = exp2f(q[kD] - base);
            l += c * q[kD + 1];
            x += c * q[tid];
        }
        o[g * kD + tid] = (uint16_t)(pack_bf16x2(x / l, 0.f) & 0xFFFFu);
    }
}

int splits(int32_t R, int32_t Hq) { return max(1, min(64, 4096 / (R * Hq))); }

}  // namespace

namespace w12i {

size_t attn_ws_bytes(int32_t R, int32_t Hq, int32_t H, int32_t n_req, int num_sms)
{
    (void)H;
    (void)n_req;
    (void)num_sms;
    return (size_t)(R * Hq + 4096) * 1 * (kD + 2) * 4;
}

int launch_attn(const AttnArgs &a, void *stream)
{
    AttnParams p{};
    p.H = a.H;
    p.Hq = a.Hq;
    p.G = a.Hq / a.H;
    p.bt = a.bt;
    p.n_blocks = a.n_blocks;
    p.max_blocks = a.max_blocks;
    p.n_req = a.n_req;
    p.R = a.R;
    p.S = splits(a.R, a.Hq);
    p.q_stride = a.q_stride;
    p.k_stride = a.k_stride;
    p.v_stride = a.v_stride;
    p.kc = a.kc;
    p.vc = a.vc;
    p.ks = a.ks;
    p.vs = a.vs;
    p.table = a.table;
    p.len = a.len;
    p.off = a.off;
    p.parent = a.parent;
    p.req = a.req;
    p.depth = a.depth;
    p.q = a.q;
    p.k = a.k;
    p.v = a.v;
    p.rope = a.rope;
    p.scale2 = a.scale * kLog2e;
    p.out = a.out;
    p.part = static_cast<float *>(a.work);
    p.status = a.status;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    k_attn_part<<<dim3(a.R * a.Hq, p.S), 128, 0, st>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return (int)e;
    const int smem = (kPath * (2 * kD + 1) + p.G * (kD + kPath)) * 4;
    e = cudaFuncSetAttribute(k_attn_join, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return (int)e;
    k_attn_join<<<dim3(a.R, a.H), 128, smem, st>>>(p);
    return (int)cudaGetLastError();
}

}  // namespace w12i
