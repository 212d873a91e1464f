// Verification of drafted tokens against the target's probabilities, from
// given random numbers.
//
// Mathematics.  Row i's target distribution is p = softmax(z / T).  Its
// children in row order are accepted by rejection sampling: child c with token
// x stands if u_accept[c] q(x) < p(x); if not, p becomes max(0, p - q) / sum and
// the next child is tried.  When none stands, the row's token is drawn from
// what p has become by the inverse CDF at u_sample[i].  With a deterministic
// drafter (no q) that reduces to drawing from p and keeping the child that has
// the drawn token.  Either way each row emits one token distributed as p.
//
// Every sum over the vocabulary is a sum of whole numbers floor(e 2^40) of the
// FP32 weights e <= 1: it does not depend on the order or the split, so a row's
// token does not change with the batch, the cluster size or the thread count,
// and inverse-CDF boundaries are exact.  (Weights under 2^-40 of the largest
// are never drawn.)
//
// A cluster of CTAs shares a row: each holds its slice of the weights in
// shared memory, so the logits are read from memory once; maxima and sums
// cross the cluster through distributed shared memory.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "w12_device.cuh"
#include "w12_kv.cuh"

namespace {

namespace cg = cooperative_groups;
using namespace w12d;
using namespace w12i;
typedef unsigned long long u64;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kMaxSlice = 49152;               // weights of one CTA: 192 KB
constexpr float kUnit = 1099511627776.f;       // 2^40

struct SampleParams {
    const void *logits;
    int64_t stride, draft_stride;
    const float *temperature, *draft_p, *u_accept, *u_sample;
    int32_t vocab, slice, sub;                 // tokens; of one CTA; of one warp
    int32_t R, n_req;
    const int32_t *parent, *token, *req, *off;
    int32_t *row_tok;
    float *row_logp;
    int32_t *status;
};

// floor(a 2^40) for 0 <= a <= 1 (and a few units above)
__device__ __forceinline__ u64 fixed40(float a)
{
    const uint32_t u = __float_as_uint(a);
    const int s = (int)(u >> 23) - 110;        // a = m 2^(e - 150): m 2^(e - 110)
    const u64 m = (u & 0x7FFFFFu) | 0x800000u;
    return s >= 0 ? m << s : (s > -24 ? m >> -s : 0ull);
}

__device__ __forceinline__ float weight_of(u64 total) { return __fmul_rn(__ull2float_rn(total), 1.f / kUnit); }

// larger float first, then the lower index (NaN is never entered)
__device__ __forceinline__ u64 max_key(float z, int v)
{
    const uint32_t b = __float_as_uint(z);
    const uint32_t o = b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
    return ((u64)o << 32) | (uint32_t)~v;
}

__device__ __forceinline__ u64 warp_sum(u64 x)
{
#pragma unroll
    for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    return x;
}

template <bool kF32>
__device__ __forceinline__ float logit(const void *row, int64_t v)
{
    return kF32 ? __ldg(static_cast<const float *>(row) + v)
                : bf16_f32(__ldg(static_cast<const unsigned short *>(row) + v));
}

struct Shared {
    u64 key[kMaxCluster];                      // written by every CTA of the cluster
    u64 total[2][kMaxCluster];
    u64 wkey[kWarps], wsum[kWarps];
    int32_t kids[kMaxBudget];
    int32_t n_kids;
};

template <bool kF32>
__global__ void __launch_bounds__(kThreads) k_sample_rows(const SampleParams p)
{
    extern __shared__ __align__(16) float w[];  // the slice's weights
    __shared__ Shared s;
    cg::cluster_group cl = cg::this_cluster();
    cl.barrier_arrive();                        // waited for before the first write to another CTA
    const int C = (int)cl.num_blocks(), rank = (int)cl.block_rank();
    const int row = blockIdx.x / C;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int v0 = rank * p.slice;
    const int n = max(0, min(p.slice, p.vocab - v0));
    const int lo = min(n, warp * p.sub), hi = min(n, lo + p.sub);   // this warp's weights, in order
    const void *zr = kF32 ? static_cast<const void *>(static_cast<const float *>(p.logits) + row * p.stride)
                          : static_cast<const void *>(static_cast<const uint16_t *>(p.logits) + row * p.stride);
    const float *qr = p.draft_p ? p.draft_p + row * p.draft_stride : nullptr;
    const int r = p.req[row];
    const bool row_ok = r >= 0 && r < p.n_req;
    if (!row_ok && tid == 0 && rank == 0) atomicCAS(p.status, 0, (int32_t)W12_E_INVAL);
    const float temp = row_ok && p.temperature ? p.temperature[r] : 1.f;
    const bool greedy = !(temp > 0.f);
    const float inv_t = greedy ? 1.f : __fdiv_rn(1.f, temp);

    // ---- z = logit / T and its maximum (lowest index on ties; NaN counts as -inf)
    u64 key = 0;
    for (int i = lo + lane; i < hi; i += 32) {
        float z = logit<kF32>(zr, v0 + i);
        if (z != z) z = -INFINITY;
        if (!greedy) z = __fmul_rn(z, inv_t);
        w[i] = z;
        const u64 k = max_key(z, v0 + i);
        key = k > key ? k : key;
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) {
        const u64 o = __shfl_xor_sync(0xffffffffu, key, d);
        key = o > key ? o : key;
    }
    if (lane == 0) s.wkey[warp] = key;
    // children of the row, in row order
    if (warp == 0 && qr) {
        int cnt = 0;
        const int end = row_ok ? min(p.R, p.off[r + 1]) : 0;
        for (int j0 = row + 1; j0 < end; j0 += 32) {
            const bool kid = j0 + lane < end && p.parent[j0 + lane] == row;
            const unsigned b = __ballot_sync(0xffffffffu, kid);
            if (kid) s.kids[cnt + __popc(b & ((1u << lane) - 1u))] = j0 + lane;
            cnt += __popc(b);
        }
        if (lane == 0) s.n_kids = cnt;
    }
    __syncthreads();
    cl.barrier_wait();
    if (warp == 0) {
        key = lane < kWarps ? s.wkey[lane] : 0;
#pragma unroll
        for (int d = 16; d; d >>= 1) {
            const u64 o = __shfl_xor_sync(0xffffffffu, key, d);
            key = o > key ? o : key;
        }
        if (lane < C) cl.map_shared_rank(s.key, lane)[rank] = key;
    }
    cl.sync();
    key = s.key[0];
    for (int c = 1; c < C; ++c) key = s.key[c] > key ? s.key[c] : key;
    const uint32_t ob = (uint32_t)(key >> 32);
    const float m = __uint_as_float(ob & 0x80000000u ? ob & 0x7FFFFFFFu : ~ob);
    const int top = (int)~(uint32_t)key;
    if (!(m > -INFINITY) || !row_ok) {          // nothing can be drawn from this row
        if (rank == 0 && tid == 0) {
            p.row_tok[row] = -1;
            if (p.row_logp) p.row_logp[row] = -INFINITY;
        }
        return;                                 // uniform over the cluster, and nobody reads another's memory any more
    }

    // ---- weights exp(z - m) and their sums
    u64 sum = 0;
    for (int i = lo + lane; i < hi; i += 32) {
        const float z = w[i];
        float e = z == m ? 1.f : expf(__fsub_rn(z, m));
        if (greedy) e = v0 + i == top ? 1.f : 0.f;
        w[i] = e;
        sum += fixed40(e);
    }
    int buf = 0;
    // sums over warps, CTA and cluster; the CTA's weights are complete after it
    auto totals = [&](u64 x) -> u64 {
        x = warp_sum(x);
        if (lane == 0) s.wsum[warp] = x;
        __syncthreads();
        if (warp == 0) {
            const u64 t = warp_sum(lane < kWarps ? s.wsum[lane] : 0ull);
            if (lane < C) cl.map_shared_rank(s.total[buf], lane)[rank] = t;
        }
        cl.sync();
        u64 t = 0;
        for (int c = 0; c < C; ++c) t += s.total[buf][c];
        return t;
    };
    u64 total = totals(sum);
    const float first = weight_of(total);
    int took = -1;
    if (qr) {
        const int n_kids = s.n_kids;
        for (int c = 0; c < n_kids; ++c) {
            const int kid = s.kids[c], x = p.token[kid];
            if (x < 0 || x >= p.vocab) continue;                   // not a token: it cannot be accepted
            const int owner = x / p.slice;
            const float ax = cl.map_shared_rank(w, owner)[x - owner * p.slice];
            const float inv = __fdiv_rn(1.f, weight_of(total));
            if (__fmul_rn(p.u_accept[kid], __ldg(qr + x)) < __fmul_rn(ax, inv)) {
                took = kid;
                break;
            }
            u64 left = 0;
            for (int i = lo + lane; i < hi; i += 32)
                left += fixed40(fmaxf(__fsub_rn(__fmul_rn(w[i], inv), __ldg(qr + v0 + i)), 0.f));
            const u64 keep = s.wsum[warp];
            buf ^= 1;
            left = totals(left);
            if (left == 0) {                                        // p = q: p stays (and so do its sums)
                if (lane == 0) s.wsum[warp] = keep;
                buf ^= 1;
                cl.sync();                                          // every CTA has read the sums it leaves
                continue;
            }
            total = left;
            for (int i = lo + lane; i < hi; i += 32)
                w[i] = fmaxf(__fsub_rn(__fmul_rn(w[i], inv), __ldg(qr + v0 + i)), 0.f);
            cl.sync();
        }
    }
    // ---- the row's token
    int tok = -1;
    if (took >= 0) {
        if (rank == 0 && tid == 0) tok = p.token[took];
    } else {
        u64 at = (u64)__dmul_rn((double)p.u_sample[row], (double)total);
        at = at < total ? at : total - 1;
        u64 before = 0;
        for (int c = 0; c < rank; ++c) before += s.total[buf][c];
        const u64 mine = s.total[buf][rank];
        if (at >= before && at < before + mine) {
            u64 t = at - before;
            int wi = 0;
            while (wi < kWarps - 1 && t >= s.wsum[wi]) t -= s.wsum[wi++];
            if (warp == wi) {
                for (int i0 = lo; i0 < hi; i0 += 32) {
                    const int i = i0 + lane;
                    const u64 x = i < hi ? fixed40(w[i]) : 0ull;
                    u64 incl = x;
#pragma unroll
                    for (int d = 1; d < 32; d <<= 1) {
                        const u64 o = __shfl_up_sync(0xffffffffu, incl, d);
                        if (lane >= d) incl += o;
                    }
                    const unsigned b = __ballot_sync(0xffffffffu, incl > t);
                    if (b) {
                        if (lane == __ffs(b) - 1) tok = v0 + i;
                        break;
                    }
                    t -= __shfl_sync(0xffffffffu, incl, 31);
                }
            }
        }
    }
    if (tok >= 0) {
        p.row_tok[row] = tok;
        if (p.row_logp) {
            float z = logit<kF32>(zr, tok);
            if (z != z) z = -INFINITY;
            z = greedy ? (tok == top ? 0.f : -INFINITY) : __fmul_rn(z, inv_t);
            p.row_logp[row] = z == m || greedy ? (greedy ? z : __fsub_rn(0.f, logf(first)))
                                               : __fsub_rn(__fsub_rn(z, m), logf(first));
        }
    }
    cl.sync();                                  // no CTA leaves while another may read its weights
}

// The accepted path: from the root to the child that carries the row's token,
// the first such child in row order, as far as there is one.  One warp per
// request; the request's rows are read once, the walk runs in shared memory.
__global__ void __launch_bounds__(128) k_sample_path(const int32_t *parent, const int32_t *token, const int32_t *off,
                                                     int32_t R, int32_t n_req, int32_t p_max, const int32_t *row_tok,
                                                     int32_t *acc_tok, int32_t *acc_len, int32_t *acc_node)
{
    __shared__ int32_t s_next[4][kMaxBudget];
    const int lane = threadIdx.x & 31, wi = threadIdx.x >> 5;
    const int r = blockIdx.x * 4 + wi;
    if (r >= n_req) return;
    int32_t *next = s_next[wi];
    const int lo = off[r], hi = off[r + 1];
    int32_t *out = acc_tok + (int64_t)r * (p_max + 1);
    for (int i = lane; i <= p_max; i += 32) out[i] = -1;
    if (lo < 0 || hi > R || lo >= hi || hi - lo > kMaxBudget) {
        if (lane == 0) {
            acc_len[r] = 0;
            if (acc_node) acc_node[r] = -1;
        }
        return;
    }
    const int rows = hi - lo;
    for (int j = lane; j < rows; j += 32) next[j] = kMaxBudget;
    pdl_wait();
    __syncwarp();
    for (int j = lane; j < rows; j += 32) {
        const int q = parent[lo + j] - lo;
        if (q >= 0 && q < j && row_tok[lo + q] == token[lo + j]) atomicMin(&next[q], j);
    }
    __syncwarp();
    if (lane == 0) {
        int cur = 0, n = 0;
        while (n < p_max && next[cur] < rows) {
            out[n++] = row_tok[lo + cur];
            cur = next[cur];
        }
        out[n] = row_tok[lo + cur];
        acc_len[r] = n + 1;
        if (acc_node) acc_node[r] = lo + cur;
    }
}

}  // namespace

namespace w12i {

int64_t sample_max_vocab() { return (int64_t)kMaxCluster * kMaxSlice; }

int launch_sample(const SampleArgs &a, void *stream)
{
    SampleParams p{};
    p.logits = a.logits;
    p.stride = a.stride;
    p.draft_stride = a.draft_stride;
    p.temperature = a.temperature;
    p.draft_p = a.draft_p;
    p.u_accept = a.u_accept;
    p.u_sample = a.u_sample;
    p.vocab = (int32_t)a.vocab;
    p.R = a.R;
    p.n_req = a.n_req;
    p.parent = a.parent;
    p.token = a.token;
    p.req = a.req;
    p.off = a.off;
    p.row_tok = a.row_tok;
    p.row_logp = a.row_logp;
    p.status = a.status;
    // as many CTAs to a row as leave each of them 2048 weights
    int c = 1;
    while (c < kMaxCluster && a.vocab > 2048 * c) c *= 2;
    p.sub = (int32_t)((a.vocab + (int64_t)c * kWarps - 1) / ((int64_t)c * kWarps) + 31) / 32 * 32;
    p.slice = p.sub * kWarps;
    const size_t smem = (size_t)p.slice * 4;
    const void *f = a.f32 ? (const void *)k_sample_rows<true> : (const void *)k_sample_rows<false>;
    cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return (int)e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(a.R * c));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)c;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = a.f32 ? cudaLaunchKernelEx(&cfg, k_sample_rows<true>, p) : cudaLaunchKernelEx(&cfg, k_sample_rows<false>, p);
    if (e != cudaSuccess || !a.acc_tok) return (int)e;
    cudaLaunchConfig_t cf{};
    cf.gridDim = dim3((unsigned)((a.n_req + 3) / 4));
    cf.blockDim = dim3(128);
    cf.stream = cfg.stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cf.attrs = at;
    cf.numAttrs = 1;
    return (int)cudaLaunchKernelEx(&cf, k_sample_path, a.parent, a.token, a.off, a.R, a.n_req, a.p_max,
                                   (const int32_t *)a.row_tok, a.acc_tok, a.acc_len, a.acc_node);
}

}  // namespace w12i
