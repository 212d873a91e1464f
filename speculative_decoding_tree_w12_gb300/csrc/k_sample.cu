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
// shared memory.  Weights are never stored: a pass makes them from the logits
// (16 bytes at a time; from L2 after the first pass, or from registers where
// few rows leave room), so a row costs one read of the logits from memory, one
// more pass for the sums, and one with the drafter's probabilities only where a
// child is rejected.  The token is found by the sums alone down to one warp's
// stretch of the row, which that warp goes through again in order.  What bounds
// many rows is the issue rate of the sums' pass, some 16 instructions a token,
// half of them expf.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

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

struct SampleParams {
    const void *logits;
    int64_t stride, draft_stride;
    const float *temperature, *draft_p, *u_accept, *u_sample;
    int32_t vocab, sub;                        // tokens; 16-byte pieces of the row of one warp
    int32_t R, n_req;
    const int32_t *parent, *token, *req, *off;
    int32_t *row_tok;
    float *row_logp;
    int32_t *acc_tok, *acc_len, *acc_node;     // acc_tok null: rows only
    int32_t p_max;
    int32_t *done, *status;                    // rows written so far
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

// the larger, or NaN
__device__ __forceinline__ float max_nan(float a, float b)
{
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ float max_nan(float a, float b, float c)
{
    float d;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
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
    u64 wsum[2][kWarps];
    int32_t kids[kMaxBudget];
    float inv[kMaxBudget];                     // of the rejections so far
    int32_t n_kids;
};

// The accepted path of request r: from the root to the first child in row order
// that carries the row's token, as far as there is one.  One warp.
__device__ void accept_path(const SampleParams &p, int r, int lane)
{
    const int lo = p.off[r], hi = p.off[r + 1];
    int32_t *out = p.acc_tok + (int64_t)r * (p.p_max + 1);
    int n = 0, cur = -1;
    if (lo >= 0 && hi <= p.R && lo < hi) {
        cur = lo;
        for (;;) {
            const int want = __ldcg(p.row_tok + cur);
            if (lane == 0) out[n] = want;
            ++n;
            int next = -1;
            if (n <= p.p_max)
                for (int j0 = cur + 1; j0 < hi && next < 0; j0 += 32) {
                    const int j = j0 + lane;
                    const unsigned b = __ballot_sync(0xffffffffu, j < hi && p.parent[j] == cur && p.token[j] == want);
                    if (b) next = j0 + __ffs(b) - 1;
                }
            if (next < 0) break;
            cur = next;
        }
    }
    for (int i = n + lane; i <= p.p_max; i += 32) out[i] = -1;
    if (lane == 0) {
        p.acc_len[r] = n;
        if (p.acc_node) p.acc_node[r] = cur;
    }
}

// After a CTA's thread has written the row's token: the CTA that writes the
// last row's goes on to the accepted paths.  (The count goes back to zero for
// the next launch.)
__device__ __forceinline__ void row_done(const SampleParams &p)
{
    if (!p.acc_tok) return;
    __shared__ int32_t s_last;
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        s_last = atomicAdd(p.done, 1) == p.R - 1;
    }
    __syncthreads();
    if (!s_last) return;
    __threadfence();
    if (threadIdx.x == 0) *p.done = 0;
    for (int r = threadIdx.x >> 5; r < p.n_req; r += kWarps) accept_path(p, r, threadIdx.x & 31);
}

// kDraft: with the drafter's probabilities.  kHold: a thread's first kHeld
// pieces stay in registers from the maximum to the sums.
template <bool kF32, bool kDraft, bool kHold>
__global__ void __launch_bounds__(kThreads, kHold ? 2 : kDraft ? 3 : 4) k_sample_rows(const SampleParams p)
{
    constexpr int kPer = Row<kF32>::kPer, kHeld = kHold ? (kF32 ? 10 : 5) : 0;
    __shared__ Shared s;
    cg::cluster_group cl = cg::this_cluster();
    cl.barrier_arrive();                        // waited for before the first write to another CTA
    const int C = (int)cl.num_blocks(), rank = (int)cl.block_rank();
    const int row = blockIdx.x / C;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const Row<kF32> z(p.logits, row * p.stride, p.vocab);
    const int pieces = (z.shift + p.vocab + kPer - 1) / kPer;
    const int lo = min(pieces, (rank * kWarps + warp) * p.sub), hi = min(pieces, lo + p.sub);   // this warp's pieces, in order
    const float *qr = kDraft ? p.draft_p + row * p.draft_stride : nullptr;
    const int r = p.req[row];
    const bool row_ok = r >= 0 && r < p.n_req;
    if (!row_ok && tid == 0 && rank == 0) atomicCAS(p.status, 0, (int32_t)W12_E_INVAL);
    const float temp = row_ok && p.temperature ? p.temperature[r] : 1.f;
    const bool greedy = !(temp > 0.f);
    const float inv_t = greedy ? 1.f : __fdiv_rn(1.f, temp);

    // ---- the largest logit, and whether there is a NaN
    uint4 held[kHold ? kHeld : 1];
    float m = -INFINITY;
    auto larger = [&](const uint4 &x) {
#pragma unroll
        for (int i = 0; i < kPer; i += 2) m = max_nan(m, Row<kF32>::get(x, i), Row<kF32>::get(x, i + 1));
    };
    if (kHold) {
#pragma unroll
        for (int k = 0; k < kHeld; ++k)
            if (lo + k * 32 + lane < hi) held[k] = z.piece(lo + k * 32 + lane);
#pragma unroll
        for (int k = 0; k < kHeld; ++k)
            if (lo + k * 32 + lane < hi) larger(held[k]);
    }
#pragma unroll 4
    for (int v = lo + kHeld * 32 + lane; v < hi; v += 32) larger(z.piece(v));
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
    bool started = false;
    auto cluster_max = [&]() {                  // of m, over the cluster
#pragma unroll
        for (int d = 16; d; d >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, d));
        if (lane == 0) s.wtop[warp] = m;
        __syncthreads();
        if (!started) cl.barrier_wait();
        started = true;
        if (warp == 0) {
            m = s.wtop[lane & (kWarps - 1)];
#pragma unroll
            for (int d = kWarps / 2; d; d >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, d));
            if (lane < C) cl.map_shared_rank(s.top, lane)[rank] = m;
        }
        cl.sync();
        m = s.top[0];
        for (int c = 1; c < C; ++c) m = max_nan(m, s.top[c]);
    };
    cluster_max();
    // NaN counts as -inf; rows that have one, or +inf, take the careful way from here on
    bool careful = m == INFINITY;
    if (m != m) {
        careful = true;
        m = -INFINITY;
        for (int v = lo + lane; v < hi; v += 32) {
            const uint4 x = z.piece(v);
#pragma unroll
            for (int i = 0; i < kPer; ++i) m = fmaxf(m, Row<kF32>::get(x, i));
        }
        cl.sync();                              // every CTA has read the last maxima
        cluster_max();
    }
    if (!(m > -INFINITY) || !row_ok) {          // nothing can be drawn from this row
        if (rank == 0) {
            if (tid == 0) {
                p.row_tok[row] = -1;
                if (p.row_logp) p.row_logp[row] = -INFINITY;
            }
            row_done(p);
        }
        return;                                 // uniform over the cluster, and nobody reads another's memory any more
    }
    if (greedy) {                               // the largest logit, the lowest token of equals, whatever the draft
        int top = p.vocab;
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
            top = __reduce_min_sync(0xffffffffu, __float_as_int(s.wtop[lane & (kWarps - 1)]));
            if (lane == 0) cl.map_shared_rank(s.first, 0)[rank] = top;
        }
        cl.sync();
        if (rank == 0) {
            if (tid == 0) {
                for (int c = 0; c < C; ++c) top = min(top, s.first[c]);
                p.row_tok[row] = top;
                if (p.row_logp) p.row_logp[row] = 0.f;
            }
            row_done(p);
        }
        return;
    }
    m = __fmul_rn(m, inv_t);                    // of z = logit / T: scaling by a positive number keeps the order

    // ---- weights exp(z - m)
    auto one = [&](float x) -> float {
        if (!careful) return expf(__fsub_rn(__fmul_rn(x, inv_t), m));
        const float y = __fmul_rn(x, inv_t);
        return y == m ? 1.f : y < m ? expf(__fsub_rn(y, m)) : 0.f;       // (a NaN is neither)
    };
    const u64 inv2 = pair(inv_t, inv_t), neg2 = pair(-m, -m);
    // the weights of tokens i and i + 1 of a piece
    auto two = [&](const uint4 &x, int i) -> u64 {
        const float a = Row<kF32>::get(x, i), b = Row<kF32>::get(x, i + 1);
        if (careful) return pair(one(a), one(b));
        const float2 d = unpair(add2(mul2(pair(a, b), inv2), neg2));
        return pair(expf(d.x), expf(d.y));
    };
    // what is left of a weight after the rejections so far
    int rounds = 0;
    auto rest = [&](float a, float q) -> float {
        for (int k = 0; k < rounds; ++k) a = fmaxf(__fsub_rn(__fmul_rn(a, s.inv[k]), q), 0.f);
        return a;
    };
    const bool q_even = kDraft && ((reinterpret_cast<uintptr_t>(qr) - 4 * z.shift) & 15) == 0;   // its pieces lie on 16 bytes too
    struct Q {                                  // the drafter's probabilities of a piece, in pairs
        u64 q[kPer / 2];
    };
    auto drafts = [&](int v) -> Q {
        Q r;
        const int t0 = v * kPer - z.shift;
        if (q_even && t0 >= 0 && t0 + kPer <= p.vocab) {
#pragma unroll
            for (int i = 0; i < kPer; i += 4) {
                const float4 f = __ldg(reinterpret_cast<const float4 *>(qr + t0 + i));
                r.q[i / 2] = pair(f.x, f.y);
                r.q[i / 2 + 1] = pair(f.z, f.w);
            }
        } else {
#pragma unroll
            for (int i = 0; i < kPer; i += 2) {
                float f[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) f[k] = t0 + i + k >= 0 && t0 + i + k < p.vocab ? __ldg(qr + t0 + i + k) : 2.f;
                r.q[i / 2] = pair(f[0], f[1]);
            }
        }
        return r;
    };
    // a piece's weights, in pairs, after the rejections so far
    auto weights = [&](const uint4 &x, const Q &q, u64 (&e)[kPer / 2]) {
#pragma unroll
        for (int i = 0; i < kPer; i += 2) e[i / 2] = two(x, i);
        if (kDraft)
            for (int k = 0; k < rounds; ++k) {
                const u64 inv = pair(s.inv[k], s.inv[k]);
#pragma unroll
                for (int i = 0; i < kPer / 2; ++i) {
                    const float2 a = unpair(fma2(q.q[i], pair(-1.f, -1.f), mul2(e[i], inv)));
                    e[i] = pair(fmaxf(a.x, 0.f), fmaxf(a.y, 0.f));
                }
            }
    };
    int buf = 0;
    // sums over warps, CTA and cluster
    auto totals = [&](u64 x) -> u64 {
        x = warp_sum(x);
        if (lane == 0) s.wsum[buf][warp] = x;
        __syncthreads();
        if (warp == 0) {
            const u64 t = warp_sum(lane < kWarps ? s.wsum[buf][lane] : 0ull);
            if (lane < C) cl.map_shared_rank(s.total[buf], lane)[rank] = t;
        }
        cl.sync();
        u64 t = 0;
        for (int c = 0; c < C; ++c) t += s.total[buf][c];
        return t;
    };
    Sum40 sum;
    auto weigh = [&](const uint4 &x) {
#pragma unroll
        for (int i = 0; i < kPer; i += 2) sum.add(two(x, i));
    };
    if (kHold) {
#pragma unroll
        for (int k = 0; k < kHeld; ++k)
            if (lo + k * 32 + lane < hi) weigh(held[k]);
    }
#pragma unroll 2
    for (int v = lo + kHeld * 32 + lane; v < hi; v += 32) weigh(z.piece(v));
    u64 total = totals(sum.get());
    const float mass = weight_of(total);
    int took = -1;
    if (kDraft) {
        const int n_kids = s.n_kids;
        for (int c = 0; c < n_kids; ++c) {
            const int kid = s.kids[c], x = p.token[kid];
            if (x < 0 || x >= p.vocab) continue;                   // not a token: it cannot be accepted
            const float q = __ldg(qr + x), a = rest(one(z.token(x)), q), inv = __fdiv_rn(1.f, weight_of(total));
            if (__fmul_rn(p.u_accept[kid], q) < __fmul_rn(a, inv)) {
                took = kid;
                break;
            }
            __syncthreads();                                        // (everyone is done with the last entry)
            if (tid == 0) s.inv[rounds] = inv;
            __syncthreads();
            ++rounds;
            Sum40 left;
            if (lo + lane < hi) {                                   // the next piece is on its way while one is summed
                uint4 y = z.piece(lo + lane);
                Q q = drafts(lo + lane);
                for (int v = lo + lane; v < hi; v += 32) {
                    const uint4 y0 = y;
                    const Q q0 = q;
                    if (v + 32 < hi) {
                        y = z.piece(v + 32);
                        q = drafts(v + 32);
                    }
                    u64 e[kPer / 2];
                    weights(y0, q0, e);
#pragma unroll
                    for (int i = 0; i < kPer / 2; ++i) left.add(e[i]);
                }
            }
            buf ^= 1;
            const u64 t = totals(left.get());
            if (t) {
                total = t;
            } else {                                                // p = q: p stays, and so do its sums
                --rounds;
                buf ^= 1;
                cl.sync();                                          // every CTA has read the sums it leaves
            }
        }
    }
    // ---- the row's token
    int tok = -1;
    bool writes = took >= 0 && rank == 0;       // this CTA has the token
    if (took >= 0) {
        if (writes && tid == 0) tok = p.token[took];
    } else {
        u64 at = (u64)__dmul_rn((double)p.u_sample[row], (double)total);
        at = at < total ? at : total - 1;
        u64 before = 0;
        for (int c = 0; c < rank; ++c) before += s.total[buf][c];
        const u64 mine = s.total[buf][rank];
        if (at >= before && at < before + mine) {
            writes = true;
            u64 t = at - before;
            int wi = 0;
            while (wi < kWarps - 1 && t >= s.wsum[buf][wi]) t -= s.wsum[buf][wi++];
            if (warp == wi) {
                for (int v0 = lo; v0 < hi; v0 += 32) {
                    const int v = v0 + lane, t0 = v * kPer - z.shift;
                    u64 e[kPer / 2];
                    Sum40 piece;
                    if (v < hi) {
                        Q q;
                        if (kDraft && rounds) q = drafts(v);
                        weights(z.piece(v), q, e);
#pragma unroll
                        for (int i = 0; i < kPer / 2; ++i) piece.add(e[i]);
                    }
                    const u64 x = piece.get();
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
                                const float2 f = unpair(e[k / 2]);
                                c += fixed40(k & 1 ? f.y : f.x);
                                if (c <= t) i = k + 1;
                            }
                            tok = t0 + i;
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
            p.row_logp[row] = __fsub_rn(x == m ? 0.f : __fsub_rn(x, m), logf(mass));
        }
    }
    if (writes) row_done(p);
}

}  // namespace

namespace w12i {

// (a thread's own sums of whole numbers stay under 2^32 up to 4096 tokens of its own)
int64_t sample_max_vocab() { return (int64_t)kThreads * 2048; }

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
    p.acc_tok = a.acc_tok;
    p.acc_len = a.acc_len;
    p.acc_node = a.acc_node;
    p.p_max = a.p_max;
    p.done = a.done;
    p.status = a.status;
    // CTAs of a row: up to 8 of 2048 tokens or more each, so that the waves of
    // them, each as long as its stretch and some 16384 tokens' worth of barriers,
    // take least (192 rows of 151936 tokens: 43 us with 8 CTAs to a row, three
    // waves, and 36 us with 3, one wave).  With no more than two to an SM, half
    // the registers of an SM hold the row between its two passes.
    const int64_t slots = (a.draft_p ? 3ll : 4ll) * a.num_sms;
    int c = 1;
    int64_t best = INT64_MAX;
    for (int i = 1; i <= kMaxCluster && (i == 1 || a.vocab > 2048 * (i - 1)); ++i) {
        const int64_t t = ((int64_t)a.R * i + slots - 1) / slots * (a.vocab / i + 16384);
        if (t < best) best = t, c = i;
    }
    const bool hold = (int64_t)a.R * c <= 2ll * a.num_sms;
    const int per = a.f32 ? 4 : 8;
    const int64_t pieces = (a.vocab + per - 1) / per + 1;         // one more where the row starts inside a piece
    p.sub = (int32_t)((pieces + (int64_t)c * kWarps - 1) / ((int64_t)c * kWarps));
    cudaError_t e = cudaSuccess;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)c;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(a.R * c));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    auto go = [&](auto kernel) { e = cudaLaunchKernelEx(&cfg, kernel, p); };
    auto pick = [&](auto f32, auto draft) {
        if (hold) go(k_sample_rows<decltype(f32)::value, decltype(draft)::value, true>);
        else go(k_sample_rows<decltype(f32)::value, decltype(draft)::value, false>);
    };
    if (a.f32) a.draft_p ? pick(std::true_type{}, std::true_type{}) : pick(std::true_type{}, std::false_type{});
    else a.draft_p ? pick(std::false_type{}, std::true_type{}) : pick(std::false_type{}, std::false_type{});
    return (int)e;
}

}  // namespace w12i
