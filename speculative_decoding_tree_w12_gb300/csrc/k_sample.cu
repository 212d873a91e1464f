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
// A cluster of CTAs shares a row; maxima and sums cross it through distributed
// shared memory.  The logits are read 16 bytes at a time, from memory for the
// maximum and from the L1 cache for the sums (a CTA's stretch is small; held in
// registers it cost half of the warps, and with them the latency of the three
// cluster barriers); only a drafter's probabilities, which change the weights
// round by round, make the weights go to shared memory.
// The token is found by the sums alone down to one warp's stretch of the row,
// which that warp reads again in order.
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

struct SampleParams {
    const void *logits;
    int64_t stride, draft_stride;
    const float *temperature, *draft_p, *u_accept, *u_sample;
    int32_t vocab, sub;                        // tokens; 16-byte pieces of the row of one warp
    int32_t R, n_req;
    const int32_t *parent, *token, *req, *off;
    int32_t *row_tok;
    float *row_logp;
    int32_t *status;
};

// Sums of whole numbers floor(e 2^40), 0 <= e <= 1.  Adding 8 with rounding
// towards zero leaves floor(e 2^20) in the low bits of the sum, subtracting it
// again the exact rest; 2^-17 splits that the same way.  Both parts are summed
// as the bits they come in; what the added constants put there is taken off at
// the end (modulo 2^32: a thread's own sums stay under 2^32).
// Two at a time where the machine adds two at a time.
__device__ __forceinline__ u64 pair(float a, float b)
{
    u64 d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ float2 unpair(u64 d)
{
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(d));
    return f;
}
__device__ __forceinline__ u64 add2(u64 a, u64 b)
{
    u64 d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ u64 add2_rz(u64 a, u64 b)
{
    u64 d;
    asm("add.rz.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ u64 mul2(u64 a, u64 b)
{
    u64 d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ u64 fma2(u64 a, u64 b, u64 c)
{
    u64 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

struct Sum40 {
    uint32_t hi = 0, lo = 0, n = 0;
    __device__ __forceinline__ void add(u64 e)
    {
        const u64 t = add2_rz(e, pair(8.f, 8.f));
        const float2 a = unpair(t);
        hi += __float_as_uint(a.x) + __float_as_uint(a.y);
        const u64 rest = fma2(add2(t, pair(-8.f, -8.f)), pair(-1.f, -1.f), e);
        const float2 b = unpair(add2_rz(rest, pair(0x1p-17f, 0x1p-17f)));
        lo += __float_as_uint(b.x) + __float_as_uint(b.y);
        n += 2;
    }
    __device__ __forceinline__ void add(float e)
    {
        const float t = __fadd_rz(e, 8.f);
        hi += __float_as_uint(t);
        lo += __float_as_uint(__fadd_rz(__fsub_rn(e, __fsub_rn(t, 8.f)), 0x1p-17f));
        ++n;
    }
    __device__ __forceinline__ u64 get() const
    {
        return ((u64)(hi - n * __float_as_uint(8.f)) << 20) + (lo - n * __float_as_uint(0x1p-17f));
    }
};

__device__ __forceinline__ u64 fixed40(float e)
{
    Sum40 s;
    s.add(e);
    return s.get();
}

__device__ __forceinline__ float weight_of(u64 total) { return __fmul_rn(__ull2float_rn(total), 0x1p-40f); }

__device__ __forceinline__ u64 warp_sum(u64 x)
{
#pragma unroll
    for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    return x;
}

__device__ __forceinline__ float warp_max(float x)
{
#pragma unroll
    for (int d = 16; d; d >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
    return x;
}

// A row of logits as 16-byte pieces on their own boundaries: piece v holds
// tokens v kPer - shift .. ; the ends are read token by token.
template <bool kF32>
struct Row {
    static constexpr int kPer = kF32 ? 4 : 8;
    const void *base;                          // of piece 0, where the row's first token may lie `shift` tokens in
    int shift, vocab;
    __device__ Row(const void *logits, int64_t at, int n)
    {
        const char *p = static_cast<const char *>(logits) + at * (kF32 ? 4 : 2);
        shift = (int)(reinterpret_cast<uintptr_t>(p) & 15) / (kF32 ? 4 : 2);
        base = p - shift * (kF32 ? 4 : 2);
        vocab = n;
    }
    __device__ __forceinline__ float token(int v) const
    {
        return kF32 ? __ldg(static_cast<const float *>(base) + shift + v)
                    : bf16_f32(__ldg(static_cast<const unsigned short *>(base) + shift + v));
    }
    __device__ __forceinline__ uint4 piece(int v) const
    {
        const int t0 = v * kPer - shift;
        if (t0 >= 0 && t0 + kPer <= vocab) return __ldg(static_cast<const uint4 *>(base) + v);
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (kF32) {
                w[i] = t0 + i >= 0 && t0 + i < vocab ? __float_as_uint(token(t0 + i)) : 0xFF800000u;   // -inf
            } else {
                const int a = t0 + 2 * i, b = a + 1;
                const uint32_t lo = a >= 0 && a < vocab ? __float_as_uint(token(a)) >> 16 : 0xFF80u;
                const uint32_t hi = b >= 0 && b < vocab ? __float_as_uint(token(b)) >> 16 : 0xFF80u;
                w[i] = lo | (hi << 16);
            }
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    __device__ __forceinline__ static float get(const uint4 &x, int i)
    {
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
        if (kF32) return __uint_as_float(w[i]);
        return i & 1 ? bf16_hi(w[i >> 1]) : bf16_lo(w[i >> 1]);
    }
};

struct Shared {
    float top[kMaxCluster];                    // written by every CTA of the cluster
    int32_t first[kMaxCluster];
    u64 total[2][kMaxCluster];
    float wtop[kWarps];
    u64 wsum[kWarps];
    int32_t kids[kMaxBudget];
    float inv[kMaxBudget];                     // of the rounds that changed the weights
    int32_t n_kids;
};

// kDraft: with the drafter's probabilities.
template <bool kF32, bool kDraft>
__global__ void __launch_bounds__(kThreads, kDraft ? 2 : 4) k_sample_rows(const SampleParams p)
{
    constexpr int kPer = Row<kF32>::kPer;
    extern __shared__ __align__(16) float w[];  // kDraft: the slice's weights
    __shared__ Shared s;
    cg::cluster_group cl = cg::this_cluster();
    cl.barrier_arrive();                        // waited for before the first write to another CTA
    pdl_launch_dependents();
    const int C = (int)cl.num_blocks(), rank = (int)cl.block_rank();
    const int row = blockIdx.x / C;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const Row<kF32> z(p.logits, row * p.stride, p.vocab);
    const int pieces = (z.shift + p.vocab + kPer - 1) / kPer;
    const int first = rank * kWarps * p.sub;    // this CTA's first piece
    const int lo = min(pieces, first + warp * p.sub), hi = min(pieces, lo + p.sub);   // this warp's pieces, in order
    const float *qr = kDraft ? p.draft_p + row * p.draft_stride : nullptr;
    const int r = p.req[row];
    const bool row_ok = r >= 0 && r < p.n_req;
    if (!row_ok && tid == 0 && rank == 0) atomicCAS(p.status, 0, (int32_t)W12_E_INVAL);
    const float temp = row_ok && p.temperature ? p.temperature[r] : 1.f;
    const bool greedy = !(temp > 0.f);
    const float inv_t = greedy ? 1.f : __fdiv_rn(1.f, temp);

    // ---- the maximum of z = logit / T (a NaN counts as -inf)
    float m = -INFINITY;
#pragma unroll 4
    for (int v = lo + lane; v < hi; v += 32) {
        const uint4 x = z.piece(v);
#pragma unroll
        for (int i = 0; i < kPer; ++i) m = fmaxf(m, Row<kF32>::get(x, i));
    }
    m = warp_max(greedy ? m : __fmul_rn(m, inv_t));      // (scaling by a positive number keeps the order)
    if (lane == 0) s.wtop[warp] = m;
    // children of the row, in row order
    if (kDraft && warp == 0) {
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
        m = warp_max(lane < kWarps ? s.wtop[lane] : -INFINITY);
        if (lane < C) cl.map_shared_rank(s.top, lane)[rank] = m;
    }
    cl.sync();
    m = s.top[0];
    for (int c = 1; c < C; ++c) m = fmaxf(m, s.top[c]);
    if (!(m > -INFINITY) || !row_ok) {          // nothing can be drawn from this row
        if (rank == 0 && tid == 0) {
            p.row_tok[row] = -1;
            if (p.row_logp) p.row_logp[row] = -INFINITY;
        }
        return;                                 // uniform over the cluster, and nobody reads another's memory any more
    }

    // ---- weights exp(z - m) and their sums
    int top = -1;
    if (greedy) {                               // all of it on the largest logit, the lowest token of equals
        top = p.vocab;
        for (int v = lo + lane; v < hi; v += 32) {
            const uint4 x = z.piece(v);
#pragma unroll
            for (int i = kPer - 1; i >= 0; --i)
                if (Row<kF32>::get(x, i) == m) top = min(top, v * kPer - z.shift + i);
        }
        top = __reduce_min_sync(0xffffffffu, top);
        if (lane == 0) s.wtop[warp] = __int_as_float(top);
        __syncthreads();
        if (warp == 0) {
            top = __reduce_min_sync(0xffffffffu, lane < kWarps ? __float_as_int(s.wtop[lane]) : p.vocab);
            if (lane < C) cl.map_shared_rank(s.first, lane)[rank] = top;
        }
        cl.sync();
        top = s.first[0];
        for (int c = 1; c < C; ++c) top = min(top, s.first[c]);
    }
    const bool flat = greedy || m == INFINITY;
    auto weight = [&](float x, int tok) -> float {
        if (flat) return greedy ? (tok == top ? 1.f : 0.f) : (x == INFINITY ? 1.f : 0.f);
        // fmaxf also turns a NaN into a weight of nothing
        return expf(fmaxf(__fsub_rn(__fmul_rn(x, inv_t), m), -128.f));
    };
    // a piece's weights: to shared memory (kDraft), and summed
    Sum40 sum;
    auto keep4 = [&](int v, int i, float a, float b, float c, float d) {
        if (kDraft) *reinterpret_cast<float4 *>(w + (v - first) * kPer + i) = make_float4(a, b, c, d);
    };
    if (flat) {
#pragma unroll 1
        for (int v = lo + lane; v < hi; v += 32) {
            const uint4 x = z.piece(v);
#pragma unroll
            for (int i = 0; i < kPer; i += 4) {
                float e[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) e[k] = weight(Row<kF32>::get(x, i + k), v * kPer - z.shift + i + k);
                sum.add(pair(e[0], e[1]));
                sum.add(pair(e[2], e[3]));
                keep4(v, i, e[0], e[1], e[2], e[3]);
            }
        }
    } else {
        const u64 inv2 = pair(inv_t, inv_t), neg2 = pair(-m, -m);
        auto two = [&](const uint4 &x, int i) -> u64 {             // the weights of tokens i and i + 1 of a piece
            const float2 d = unpair(add2(mul2(pair(Row<kF32>::get(x, i), Row<kF32>::get(x, i + 1)), inv2), neg2));
            return pair(expf(fmaxf(d.x, -128.f)), expf(fmaxf(d.y, -128.f)));   // (a NaN becomes a weight of nothing)
        };
#pragma unroll 2
        for (int v = lo + lane; v < hi; v += 32) {
            const uint4 x = z.piece(v);
#pragma unroll
            for (int i = 0; i < kPer; i += 4) {
                const u64 a = two(x, i), b = two(x, i + 2);
                sum.add(a);
                sum.add(b);
                const float2 e = unpair(a), f = unpair(b);
                keep4(v, i, e.x, e.y, f.x, f.y);
            }
        }
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
    u64 total = totals(sum.get());
    const float mass = weight_of(total);
    int took = -1, rounds = 0;
    // what a weight becomes where a child is rejected; element i of the warp's stretch is token t0 + i
    const int t0 = lo * kPer - z.shift, n = (hi - lo) * kPer;
    float *wl = w + (lo - first) * kPer;
    if (kDraft) {
        auto residual = [&](float a, float inv, int tok) -> float {
            return tok >= 0 && tok < p.vocab ? fmaxf(__fsub_rn(__fmul_rn(a, inv), __ldg(qr + tok)), 0.f) : 0.f;
        };
        const int n_kids = s.n_kids, per_cta = kWarps * p.sub * kPer;
        for (int c = 0; c < n_kids; ++c) {
            const int kid = s.kids[c], x = p.token[kid];
            if (x < 0 || x >= p.vocab) continue;                   // not a token: it cannot be accepted
            const int owner = (x + z.shift) / per_cta;
            const float ax = cl.map_shared_rank(w, owner)[x + z.shift - owner * per_cta];
            const float inv = __fdiv_rn(1.f, weight_of(total));
            if (__fmul_rn(p.u_accept[kid], __ldg(qr + x)) < __fmul_rn(ax, inv)) {
                took = kid;
                break;
            }
            cl.sync();                                              // every CTA has read ax
            Sum40 rest;
            for (int i = lane; i < n; i += 32) {
                const float a = residual(wl[i], inv, t0 + i);
                wl[i] = a;
                rest.add(a);
            }
            const u64 keep = s.wsum[warp];
            buf ^= 1;
            const u64 left = totals(rest.get());
            if (left) {
                total = left;
                if (tid == 0) s.inv[rounds] = inv;
                ++rounds;
                continue;
            }
            // p = q: p stays, and so do its sums; the weights are made again
            if (lane == 0) s.wsum[warp] = keep;
            buf ^= 1;
            __syncthreads();
            for (int i = lane; i < n; i += 32) {
                const int tok = t0 + i;
                float a = tok >= 0 && tok < p.vocab ? weight(z.token(tok), tok) : 0.f;
                for (int k = 0; k < rounds; ++k) a = residual(a, s.inv[k], tok);
                wl[i] = a;
            }
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
                for (int v0 = lo; v0 < hi; v0 += 32) {
                    const int v = v0 + lane;
                    float e[kPer];
                    u64 x = 0;
                    if (v < hi) {
                        const uint4 y = kDraft ? make_uint4(0, 0, 0, 0) : z.piece(v);
#pragma unroll
                        for (int i = 0; i < kPer; ++i) {
                            e[i] = kDraft ? w[(v - first) * kPer + i] : weight(Row<kF32>::get(y, i), v * kPer - z.shift + i);
                            x += fixed40(e[i]);
                        }
                    }
                    u64 incl = x;
#pragma unroll
                    for (int d = 1; d < 32; d <<= 1) {
                        const u64 o = __shfl_up_sync(0xffffffffu, incl, d);
                        if (lane >= d) incl += o;
                    }
                    const unsigned b = __ballot_sync(0xffffffffu, incl > t);
                    if (b) {
                        if (lane == __ffs(b) - 1) {
                            u64 c = incl - x;
                            int i = 0;
#pragma unroll
                            for (int k = 0; k < kPer - 1; ++k) {
                                c += fixed40(e[k]);
                                if (c <= t) i = k + 1;
                            }
                            tok = v * kPer - z.shift + i;
                        }
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
            // (a NaN can only be an accepted child's)
            const float x = __fmul_rn(fmaxf(z.token(tok), -INFINITY), inv_t);
            p.row_logp[row] = greedy ? (tok == top ? 0.f : -INFINITY) : __fsub_rn(x == m ? 0.f : __fsub_rn(x, m), logf(mass));
        }
    }
    if (kDraft) cl.sync();                       // no CTA leaves while another may read its weights
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
    // as many CTAs to a row as leave each of them 2048 tokens
    int c = 1;
    while (c < kMaxCluster && a.vocab > 2048 * c) c *= 2;
    const int per = a.f32 ? 4 : 8;
    const int64_t pieces = (a.vocab + per - 1) / per + 1;         // one more where the row starts inside a piece
    p.sub = (int32_t)((pieces + (int64_t)c * kWarps - 1) / ((int64_t)c * kWarps));
    const size_t smem = a.draft_p ? (size_t)p.sub * kWarps * per * 4 : 0;
    cudaError_t e = cudaSuccess;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)c;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(a.R * c));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    auto go = [&](auto kernel) {
        if (smem) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, kernel, p);
    };
    if (a.f32) a.draft_p ? go(k_sample_rows<true, true>) : go(k_sample_rows<true, false>);
    else a.draft_p ? go(k_sample_rows<false, true>) : go(k_sample_rows<false, false>);
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
