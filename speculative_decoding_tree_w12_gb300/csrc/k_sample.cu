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
// k_sample_max and k_sample_sum go over the logits in chunks, each chunk a CTA:
// the first for the rows' maxima, the second (from L2, asked for before it has
// to wait for the maxima) for the sums of the weights of every warp's stretch.
// The CTA that completes a row finds the stretch its token lies in by these
// sums, and goes through it once more in order.  With a drafter's probabilities
// the rows whose first child was rejected are left to k_sample_draft: a cluster
// to a row, which goes over it again for every rejection.
// The CTA that completes the last row writes the accepted paths.
// The second pass takes the rows in reverse, so that logits past the L2 cache's
// size are found there as far as it reaches.
//
// What bounds it.  192 rows of 151936 BF16 tokens (58 MB) take 41 us: 7 for the
// maxima, 25 for the sums, at the issue rate of some twenty instructions a
// token, half of them expf, 8 for the last rows' draws and the paths, each a
// chain of loads.  256 FP32 rows with a drafter's probabilities (156 MB, and as
// much of the drafter's for the rows with a rejection) take 115 to 123 us: 25
// and 36 for the two passes, 50 for some 40 rejected rows, which are few to
// spread over the SMs and wait for their slowest.  One row takes 10 us, all of
// it latency.
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

constexpr int kThreads = 512;                  // k_sample_draft
constexpr int kWarps = kThreads / 32;
constexpr int kChunkThreads = 256;             // k_sample_max, k_sample_sum
constexpr int kChunkWarps = kChunkThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int64_t kMaxVocab = 1 << 20;

struct SampleParams {
    const void *logits;
    int64_t stride, draft_stride;
    const float *temperature, *draft_p, *u_accept, *u_sample;
    int32_t vocab, sub;                        // tokens; 16-byte pieces of the row of one warp of k_sample_draft
    int32_t chunks, per;                       // of a row; pieces of a thread of the two passes (a warp's stretch: 32 per)
    int32_t R, n_req;
    const int32_t *parent, *token, *req, *off;
    int32_t *row_tok;
    float *row_logp;
    int32_t *acc_tok, *acc_len, *acc_node;     // acc_tok null: rows only
    int32_t p_max;
    int32_t *status;
    // scratch
    int32_t *done, *n_left, *taken;            // rows written, left to k_sample_draft, taken there behind every cluster's first
    int32_t *arrived;                          // [R] chunks summed
    float *top;                                // [R][chunks] largest logit
    struct Left *left;                         // [R]
    u64 *sums;                                 // [R][chunks][kChunkWarps] (greedy rows: lowest token with the largest logit)
};

// a row whose first child was rejected
struct Left {
    int32_t row;
    float top;
    u64 total;
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
    // no token of pieces lo .. hi - 1 is outside the row
    __device__ __forceinline__ bool inner(int lo, int hi) const { return lo * kPer >= shift && hi * kPer - shift <= vocab; }
    __device__ __forceinline__ uint4 whole(int v) const { return __ldg(static_cast<const uint4 *>(base) + v); }
    __device__ __forceinline__ uint4 piece(int v) const                  // -inf outside the row
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
    // the lane's pieces of N * 32 from v0
    template <int N>
    __device__ __forceinline__ void load(int v0, int lane, uint4 (&x)[N]) const
    {
        if (inner(v0, v0 + N * 32)) {
#pragma unroll
            for (int j = 0; j < N; ++j) x[j] = whole(v0 + j * 32 + lane);
        } else {
#pragma unroll
            for (int j = 0; j < N; ++j) x[j] = piece(v0 + j * 32 + lane);
        }
    }
    __device__ __forceinline__ static float get(const uint4 &x, int i)
    {
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
        if (kF32) return __uint_as_float(w[i]);
        return i & 1 ? bf16_hi(w[i >> 1]) : bf16_lo(w[i >> 1]);
    }
};

// The accepted paths of requests r0, r0 + step .. (N at most): from the root
// to the first child in row order that carries the row's token, as far as there
// is one.  One warp; the first 32 rows of all N are fetched at once, and what
// is in the tree before it is known whether all rows have their tokens.
template <int N>
struct Paths {
    int lo[N], hi[N], parent[N], token[N];
};

template <int N>
__device__ __forceinline__ Paths<N> fetch_paths(const SampleParams &p, int r0, int step, int lane)
{
    Paths<N> t;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int r = r0 + i * step;
        t.lo[i] = r < p.n_req ? p.off[r] : 0;
        t.hi[i] = r < p.n_req ? p.off[r + 1] : 0;
        if (t.lo[i] < 0 || t.hi[i] > p.R) t.hi[i] = t.lo[i];
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int j = t.lo[i] + lane;
        t.parent[i] = j < t.hi[i] ? p.parent[j] : -1;
        t.token[i] = j < t.hi[i] ? p.token[j] : -1;
    }
    return t;
}

template <int N>
__device__ __forceinline__ void accept_paths(const SampleParams &p, int r0, int step, int lane, const Paths<N> &t)
{
    int drawn[N];
#pragma unroll
    for (int i = 0; i < N; ++i) drawn[i] = t.lo[i] + lane < t.hi[i] ? __ldcg(p.row_tok + t.lo[i] + lane) : -1;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int r = r0 + i * step, lo = t.lo[i], hi = t.hi[i];
        if (r >= p.n_req) break;
        int32_t *out = p.acc_tok + (int64_t)r * (p.p_max + 1);
        int n = 0, cur = -1;
        if (lo < hi) {
            cur = lo;
            for (;;) {
                const int want = cur - lo < 32 ? __shfl_sync(0xffffffffu, drawn[i], cur - lo) : __ldcg(p.row_tok + cur);
                if (lane == 0) out[n] = want;
                ++n;
                if (n > p.p_max) break;
                const int j = lo + lane;
                unsigned b = __ballot_sync(0xffffffffu, j < hi && j > cur && t.parent[i] == cur && t.token[i] == want);
                int next = b ? lo + __ffs(b) - 1 : -1;
                for (int j0 = max(cur + 1, lo + 32); j0 < hi && next < 0; j0 += 32) {
                    const int k = j0 + lane;
                    b = __ballot_sync(0xffffffffu, k < hi && p.parent[k] == cur && p.token[k] == want);
                    if (b) next = j0 + __ffs(b) - 1;
                }
                if (next < 0) break;
                cur = next;
            }
        }
        for (int k = n + lane; k <= p.p_max; k += 32) out[k] = -1;
        if (lane == 0) {
            p.acc_len[r] = n;
            if (p.acc_node) p.acc_node[r] = cur;
        }
    }
}

// After a CTA's thread has written the row's token: the CTA that writes the
// last row's goes on to the accepted paths, N of a warp at a time.
template <int N>
__device__ __forceinline__ void row_done(const SampleParams &p)
{
    if (!p.acc_tok) return;
    __shared__ int32_t s_last;
    const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
    int r = threadIdx.x >> 5;
    Paths<N> t = fetch_paths<N>(p, r, warps, lane);
    __syncthreads();
    if (p.R > 1) {
        if (threadIdx.x == 0) {
            __threadfence();
            s_last = atomicAdd(p.done, 1) == p.R - 1;
        }
        __syncthreads();
        if (!s_last) return;
        __threadfence();
    }
    for (;;) {
        accept_paths(p, r, warps, lane, t);
        r += N * warps;
        if (r >= p.n_req) break;
        t = fetch_paths<N>(p, r, warps, lane);
    }
}

// a greedy row's token: the lowest of the chunks' candidates.  One warp.
__device__ __forceinline__ void draw_greedy(const SampleParams &p, int row, int lane)
{
    int tok = INT32_MAX;
    for (int i = lane; i < p.chunks * kChunkWarps; i += 32)
        tok = min(tok, (int)__ldcg(p.sums + (int64_t)row * p.chunks * kChunkWarps + i));
    tok = __reduce_min_sync(0xffffffffu, tok);
    if (lane == 0) {
        p.row_tok[row] = tok;
        if (p.row_logp) p.row_logp[row] = 0.f;
    }
}

// ---------------------------------------------------------------------------
// what the kernels share: a row's temperature, weights and the search
// ---------------------------------------------------------------------------

struct Temper {
    float inv_t;
    bool ok, greedy;
};

__device__ __forceinline__ Temper temper(const SampleParams &p, int row)
{
    const int r = p.req[row];
    Temper t;
    t.ok = r >= 0 && r < p.n_req;
    const float T = t.ok && p.temperature ? p.temperature[r] : 1.f;
    t.inv_t = __fdiv_rn(1.f, T);
    t.greedy = !(T > 0.f) || t.inv_t == INFINITY;                       // (1 / T over the numbers' range: next to nothing)
    return t;
}

// exp(z - m), z = logit / T.  With 10^5 tokens the next boundary of the CDF is
// as near as 10^-6 of the mass, so the weights have to be as good as FP32 gives
// them: expf, the largest part of the sums' pass.  (The machine's own 2^x would
// take six instructions a token less, 192 rows 35 us instead of 40, and drew
// another token than FP32's exponentials in one row of 200.)
template <bool kF32>
struct Weigher {
    static constexpr int kPer = Row<kF32>::kPer;
    static constexpr float kLeast = -128.f;    // (also what a NaN becomes: a weight of nothing)
    float inv_t, top, m;                       // m: the largest z
    // The largest z may be no number: an infinite logit, or one of the type's
    // lowest or highest over a T under 1.  Then the logits equal to the largest
    // weigh 1 and all others nothing, as in the limit: two different ones of
    // that size lie further apart than 2^100 T.  So a row's weights never sum
    // to nothing.
    bool flat;
    __device__ Weigher(float inv_t_, float top_) : inv_t(inv_t_), top(top_), m(top_ * inv_t_), flat(!(fabsf(m) < INFINITY)) {}   // (a positive factor keeps the order)
    __device__ __forceinline__ float one(float x) const
    {
        if (flat) return x == top ? 1.f : 0.f;
        return expf(fmaxf(__fsub_rn(__fmul_rn(x, inv_t), m), kLeast));
    }
    // of a piece's tokens, in pairs; kFlat: as above
    template <bool kFlat = false>
    __device__ __forceinline__ void piece(const uint4 &x, u64 (&e)[kPer / 2]) const
    {
#pragma unroll
        for (int i = 0; i < kPer; i += 2) {
            if (kFlat) {
                e[i / 2] = pair(one(Row<kF32>::get(x, i)), one(Row<kF32>::get(x, i + 1)));
                continue;
            }
            // (a product and a difference of two would be fused, and round once)
            const float2 z = unpair(mul2(pair(Row<kF32>::get(x, i), Row<kF32>::get(x, i + 1)), pair(inv_t, inv_t)));
            e[i / 2] = pair(expf(fmaxf(__fsub_rn(z.x, m), kLeast)), expf(fmaxf(__fsub_rn(z.y, m), kLeast)));
        }
    }
    __device__ __forceinline__ void any_piece(const uint4 &x, u64 (&e)[kPer / 2]) const
    {
        if (flat) piece<true>(x, e);
        else piece(x, e);
    }
};

// The warp's token of a stretch of pieces lo .. hi - 1: the first whose weights
// up to and with it sum to more than t; -1 on all lanes but the one that has it.
// `piece(v, e)` gives a piece's weights in pairs.
template <int kPer, class Piece>
__device__ __forceinline__ int find_token(int lo, int hi, u64 t, int shift, int lane, Piece piece)
{
    for (int v0 = lo; v0 < hi; v0 += 32) {
        const int v = v0 + lane;
        u64 e[kPer / 2];
        Sum40 s;
        if (v < hi) {
            piece(v, e);
#pragma unroll
            for (int i = 0; i < kPer / 2; ++i) s.add(e[i]);
        }
        const u64 x = s.get();
        u64 incl = x;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const u64 o = __shfl_up_sync(0xffffffffu, incl, d);
            if (lane >= d) incl += o;
        }
        const unsigned b = __ballot_sync(0xffffffffu, incl > t);
        if (b) {
            if (lane != __ffs(b) - 1) return -1;
            u64 c = incl - x;
            int i = 0;
#pragma unroll
            for (int k = 0; k < kPer - 1; ++k) {
                const float2 f = unpair(e[k / 2]);
                c += fixed40(k & 1 ? f.y : f.x);
                if (c <= t) i = k + 1;
            }
            return v * kPer - shift + i;
        }
        t -= __shfl_sync(0xffffffffu, incl, 31);
    }
    return -1;
}

// where u of the mass lies
__device__ __forceinline__ u64 place(float u, u64 total)
{
    const u64 at = (u64)__dmul_rn((double)u, (double)total);
    return at < total ? at : total - 1;
}

template <bool kF32>
__device__ __forceinline__ void write_row(const SampleParams &p, int row, int tok, float logit, const Weigher<kF32> &w, u64 total)
{
    p.row_tok[row] = tok;
    if (p.row_logp) {
        // (a NaN can only be an accepted child's)
        const float x = __fmul_rn(fmaxf(logit, -INFINITY), w.inv_t);
        const float z = w.flat ? (logit == w.top ? 0.f : -INFINITY) : __fsub_rn(x, w.m);
        p.row_logp[row] = __fsub_rn(z, logf(weight_of(total)));
    }
}

__device__ __forceinline__ void write_none(const SampleParams &p, int row)
{
    p.row_tok[row] = -1;
    if (p.row_logp) p.row_logp[row] = -INFINITY;
}

// the row's largest logit, by every warp for itself
__device__ __forceinline__ float row_top(const SampleParams &p, int row, int lane)
{
    float m = -INFINITY;
    for (int c = lane; c < p.chunks; c += 32) m = fmaxf(m, __ldcg(p.top + (int64_t)row * p.chunks + c));
#pragma unroll
    for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    return m;
}

// The row's token, by one CTA: where the weights of the stretch of 32 n pieces
// from `first` sum to more than t.  Every warp takes a part of the stretch.
template <bool kF32, class Piece>
__device__ __forceinline__ void search(const SampleParams &p, int row, int first, int n, u64 t, const Row<kF32> &z, const Weigher<kF32> &w,
                                       u64 total, u64 *s_sum, Piece weigh)
{
    uint4 x;                                   // the last piece
    auto piece = [&](int v, auto &e) {
        x = z.piece(v);
        weigh(v, x, e);
    };
    constexpr int kPer = Row<kF32>::kPer;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int sub = (n + warps - 1) / warps * 32;
    const int lo = first + warp * sub, hi = min(first + 32 * n, lo + sub);
    bool mine = warp == 0;
    if (n > 1) {
        Sum40 sum;
        for (int v = lo + lane; v < hi; v += 32) {
            u64 e[kPer / 2];
            piece(v, e);
#pragma unroll
            for (int i = 0; i < kPer / 2; ++i) sum.add(e[i]);
        }
        const u64 all = warp_sum(sum.get());
        if (lane == 0) s_sum[warp] = all;
        __syncthreads();
        for (int i = 0; i < warp; ++i) {
            if (t < s_sum[i]) return;
            t -= s_sum[i];
        }
        mine = t < all;
    }
    if (!mine) return;
    const int tok = find_token<kPer>(lo, hi, t, z.shift, lane, piece);
    if (tok >= 0) {
        float logit = 0.f;
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (i == (tok + z.shift) % kPer) logit = Row<kF32>::get(x, i);
        write_row(p, row, tok, logit, w, total);
    }
}

// The sums of a row's stretches, a run of them to a thread.
struct Scan {
    u64 *sums;
    int first, end;                            // this thread's
    u64 before, mine, total;
};

__device__ __forceinline__ Scan scan_row(const SampleParams &p, int row, u64 *s_sum)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, threads = blockDim.x;
    const int n = p.chunks * kChunkWarps, run = (n + threads - 1) / threads;
    Scan c;
    c.sums = p.sums + (int64_t)row * n;
    c.first = min(n, (int)threadIdx.x * run);
    c.end = min(n, c.first + run);
    c.mine = c.total = 0;
    for (int i = c.first; i < c.end; ++i) c.mine += __ldcg(c.sums + i);
    c.before = c.mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const u64 o = __shfl_up_sync(0xffffffffu, c.before, d);
        if (lane >= d) c.before += o;
    }
    if (lane == 31) s_sum[warp] = c.before;
    c.before -= c.mine;
    __syncthreads();
    for (int i = 0; i < threads / 32; ++i) {
        if (i < warp) c.before += s_sum[i];
        c.total += s_sum[i];
    }
    __syncthreads();
    return c;
}

// A row without rejections, by one CTA: its token by the sums of the stretches.
template <bool kF32>
__device__ void draw(const SampleParams &p, int row, const Row<kF32> &z, const Weigher<kF32> &w, const Scan &c, u64 *s_sum)
{
    constexpr int kPer = Row<kF32>::kPer;
    __shared__ u64 s_rest;
    __shared__ int32_t s_at;
    u64 t = place(p.u_sample[row], c.total);
    if (t >= c.before && t - c.before < c.mine) {
        t -= c.before;
        int at = c.first;
        for (;; ++at) {
            const u64 x = __ldcg(c.sums + at);
            if (t < x) break;
            t -= x;
        }
        s_at = at;
        s_rest = t;
    }
    __syncthreads();
    search(p, row, s_at * 32 * p.per, p.per, s_rest, z, w, c.total, s_sum, [&](int, const uint4 &x, u64 (&e)[kPer / 2]) { w.any_piece(x, e); });
}

// The row's next child after row j, of those whose token is one.  One warp.
__device__ __forceinline__ int next_child(const SampleParams &p, int row, int j, int lane)
{
    const int end = min(p.R, p.off[p.req[row] + 1]);
    for (int j0 = j + 1; j0 < end; j0 += 32) {
        const int k = j0 + lane;
        const unsigned b = __ballot_sync(0xffffffffu, k < end && p.parent[k] == row && p.token[k] >= 0 && p.token[k] < p.vocab);
        if (b) return j0 + __ffs(b) - 1;
    }
    return -1;
}

// u q < p with the child's weight a of the total's
__device__ __forceinline__ bool accepted(float u, float q, float a, u64 total)
{
    return __fmul_rn(u, q) < __fmul_rn(a, __fdiv_rn(1.f, weight_of(total)));
}

// ---------------------------------------------------------------------------
// the two passes
// ---------------------------------------------------------------------------

// N: pieces in flight of a thread, a divisor of per
template <bool kF32, int N>
__global__ void __launch_bounds__(kChunkThreads, 8) k_sample_max(const SampleParams p)
{
    constexpr int kPer = Row<kF32>::kPer;
    __shared__ float s_top[kChunkWarps];
    const int row = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Row<kF32> z(p.logits, row * p.stride, p.vocab);
    const int lo = (blockIdx.x * kChunkWarps + warp) * 32 * p.per;
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        p.arrived[row] = 0;
        if (row == 0) *p.done = *p.n_left = *p.taken = 0;
    }
    pdl_launch_dependents();
    float m = -INFINITY;
    for (int k = 0; k < p.per; k += N) {
        uint4 x[N];
        z.load(lo + k * 32, lane, x);
#pragma unroll
        for (int j = 0; j < N; ++j)
#pragma unroll
            for (int i = 0; i < kPer; i += 2) m = fmaxf(fmaxf(m, Row<kF32>::get(x[j], i)), Row<kF32>::get(x[j], i + 1));
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    if (lane == 0) s_top[warp] = m;
    __syncthreads();
    if (threadIdx.x == 0) {
#pragma unroll
        for (int w = 1; w < kChunkWarps; ++w) m = fmaxf(m, s_top[w]);
        p.top[(int64_t)row * p.chunks + blockIdx.x] = m;
    }
}

template <bool kF32, int N, bool kDraft>
__global__ void __launch_bounds__(kChunkThreads, 5) k_sample_sum(const SampleParams p)
{
    constexpr int kPer = Row<kF32>::kPer;
    __shared__ int32_t s_last;
    __shared__ u64 s_sum[kChunkWarps];
    const int row = gridDim.y - 1 - blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Row<kF32> z(p.logits, row * p.stride, p.vocab);
    const int lo = (blockIdx.x * kChunkWarps + warp) * 32 * p.per;
    const Temper t = temper(p, row);
    if (kDraft) pdl_launch_dependents();
    uint4 x[N];
    z.load(lo, lane, x);
    pdl_wait();
    const float top = row_top(p, row, lane);
    const Weigher<kF32> w(t.inv_t, top);
    u64 *mine = p.sums + ((int64_t)row * p.chunks + blockIdx.x) * kChunkWarps + warp;
    if (t.greedy) {                             // the largest logit, the lowest token of equals, whatever the draft
        int tok = INT32_MAX;
        for (int k = 0;;) {
#pragma unroll
            for (int j = 0; j < N; ++j)
#pragma unroll
                for (int i = 0; i < kPer; ++i)
                    if (Row<kF32>::get(x[j], i) == top) tok = min(tok, (lo + (k + j) * 32 + lane) * kPer - z.shift + i);
            if ((k += N) >= p.per) break;
            z.load(lo + k * 32, lane, x);
        }
        tok = __reduce_min_sync(0xffffffffu, tok);
        if (lane == 0) *mine = (u64)tok;
    } else {
        Sum40 sum;
        auto stretch = [&](auto flat) {
            for (int k = 0;;) {
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    u64 e[kPer / 2];
                    w.template piece<decltype(flat)::value>(x[j], e);
#pragma unroll
                    for (int i = 0; i < kPer / 2; ++i) sum.add(e[i]);
                }
                if ((k += N) >= p.per) break;
                z.load(lo + k * 32, lane, x);
            }
        };
        if (w.flat) stretch(std::true_type{});
        else stretch(std::false_type{});
        const u64 all = warp_sum(sum.get());
        if (lane == 0) *mine = all;
    }
    // ---- the row's last CTA draws its token, or leaves it to k_sample_draft
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        s_last = atomicAdd(p.arrived + row, 1) == p.chunks - 1;
    }
    __syncthreads();
    if (!s_last) return;
    __threadfence();
    const bool first = threadIdx.x == 0;
    if (first && !t.ok) atomicCAS(p.status, 0, (int32_t)W12_E_INVAL);
    if (!(top > -INFINITY) || !t.ok) {          // nothing can be drawn from this row
        if (first) write_none(p, row);
    } else if (t.greedy) {
        if (warp == 0) draw_greedy(p, row, lane);
    } else {
        const Scan c = scan_row(p, row, s_sum);
        const int kid = kDraft ? next_child(p, row, row, lane) : -1;
        if (kid < 0) {
            draw(p, row, z, w, c, s_sum);
        } else {
            const int x = p.token[kid];
            const float logit = z.token(x);
            if (!accepted(p.u_accept[kid], __ldg(p.draft_p + row * p.draft_stride + x), w.one(logit), c.total)) {
                if (first) p.left[atomicAdd(p.n_left, 1)] = {row, top, c.total};
                return;
            }
            if (first) write_row(p, row, x, logit, w, c.total);
        }
    }
    row_done<4>(p);
}

// ---------------------------------------------------------------------------
// rejection sampling
// ---------------------------------------------------------------------------

struct Shared {
    u64 total[2][kMaxCluster];                 // written by every CTA of the cluster
    u64 wsum[2][kWarps];
    float inv[kMaxBudget];                     // of the rejections so far
    struct {
        int32_t row;
        float u, q, e;                         // its number, the drafter's probability, the weight
    } kid[kMaxBudget];                         // children, in row order
    int32_t n_kids;
    int32_t next;                              // row, of those left over; written by the cluster's first CTA
};

template <bool kF32>
__device__ __forceinline__ void reject(const SampleParams &p, Shared &s, const cg::cluster_group &cl, const Left &job)
{
    constexpr int kPer = Row<kF32>::kPer;
    const int C = (int)cl.num_blocks(), rank = (int)cl.block_rank();
    const int row = job.row;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const Row<kF32> z(p.logits, row * p.stride, p.vocab);
    const int lo = (rank * kWarps + warp) * p.sub, hi = lo + p.sub;   // this warp's pieces, in order
    const float *qr = p.draft_p + row * p.draft_stride;
    const Weigher<kF32> w(temper(p, row).inv_t, job.top);
    u64 total = job.total;
    if (warp == 0) {
        int n = 0;
        const int end = min(p.R, p.off[p.req[row] + 1]);
        for (int j0 = row + 1; j0 < end; j0 += 32) {
            const int j = j0 + lane, x = j < end && p.parent[j] == row ? p.token[j] : -1;
            const bool is = x >= 0 && x < p.vocab;                  // (what is no token cannot be accepted)
            const unsigned b = __ballot_sync(0xffffffffu, is);
            if (is) s.kid[n + __popc(b & ((1u << lane) - 1u))] = {j, p.u_accept[j], __ldg(qr + x), w.one(z.token(x))};
            n += __popc(b);
        }
        if (lane == 0) s.n_kids = n;
    }
    __syncthreads();
    const bool q_even = ((reinterpret_cast<uintptr_t>(qr) - 4 * z.shift) & 15) == 0;   // its pieces lie on 16 bytes too
    int rounds = 0;
    struct Q {                                  // the drafter's probabilities of a piece, in pairs
        u64 q[kPer / 2];
    };
    auto whole_drafts = [&](int v) -> Q {
        Q r;
#pragma unroll
        for (int i = 0; i < kPer; i += 4) {
            const float4 f = __ldg(reinterpret_cast<const float4 *>(qr + v * kPer - z.shift + i));
            r.q[i / 2] = pair(f.x, f.y);
            r.q[i / 2 + 1] = pair(f.z, f.w);
        }
        return r;
    };
    auto drafts = [&](int v) -> Q {
        Q r;
        const int t0 = v * kPer - z.shift;
#pragma unroll
        for (int i = 0; i < kPer; i += 2) {
            float f[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) f[k] = t0 + i + k >= 0 && t0 + i + k < p.vocab ? __ldg(qr + t0 + i + k) : 2.f;
            r.q[i / 2] = pair(f[0], f[1]);
        }
        return r;
    };
    // what is left of a piece's weights after the rejections so far, in pairs
    auto weights = [&](const uint4 &x, const Q &q, u64 (&e)[kPer / 2]) {
        w.any_piece(x, e);
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
            const u64 c = warp_sum(lane < kWarps ? s.wsum[buf][lane] : 0ull);
            if (lane < C) cl.map_shared_rank(s.total[buf], lane)[rank] = c;
        }
        cl.sync();
        u64 c = 0;
        for (int i = 0; i < C; ++i) c += s.total[buf][i];
        return c;
    };
    int took = -1;
    const int n_kids = s.n_kids;
    for (int c = 0; c < n_kids; ++c) {
        const auto kid = s.kid[c];
        float a = kid.e;
        for (int k = 0; k < rounds; ++k) a = fmaxf(__fsub_rn(__fmul_rn(a, s.inv[k]), kid.q), 0.f);
        if (accepted(kid.u, kid.q, a, total)) {
            took = kid.row;
            break;
        }
        __syncthreads();                                            // (everyone is done with the last entry)
        if (tid == 0) s.inv[rounds] = __fdiv_rn(1.f, weight_of(total));
        __syncthreads();
        ++rounds;
        Sum40 left;
        constexpr int kBatch = kF32 ? 2 : 1;                        // pieces in flight of a thread
        for (int v0 = lo; v0 < hi; v0 += 32 * kBatch) {
            const int n = min(kBatch, (hi - v0) / 32);
            uint4 y[kBatch];
            Q d[kBatch];
            if (q_even && z.inner(v0, v0 + n * 32)) {
#pragma unroll
                for (int j = 0; j < kBatch; ++j)
                    if (j < n) {
                        y[j] = z.whole(v0 + j * 32 + lane);
                        d[j] = whole_drafts(v0 + j * 32 + lane);
                    }
            } else {
#pragma unroll
                for (int j = 0; j < kBatch; ++j)
                    if (j < n) {
                        y[j] = z.piece(v0 + j * 32 + lane);
                        d[j] = drafts(v0 + j * 32 + lane);
                    }
            }
#pragma unroll
            for (int j = 0; j < kBatch; ++j)
                if (j < n) {
                    u64 e[kPer / 2];
                    weights(y[j], d[j], e);
#pragma unroll
                    for (int i = 0; i < kPer / 2; ++i) left.add(e[i]);
                }
        }
        buf ^= 1;
        const u64 r = totals(left.get());
        if (r) {
            total = r;
        } else {                                                    // p = q: p stays, and so do its sums
            --rounds;
            buf ^= 1;
            cl.sync();                                              // every CTA has read the sums it leaves
        }
    }
    // ---- the row's token
    bool writes = rank == 0;                                        // this CTA has it
    if (took >= 0) {
        if (writes && tid == 0) write_row(p, row, p.token[took], z.token(p.token[took]), w, job.total);
    } else if (rounds == 0) {                                       // p = q
        if (writes) draw(p, row, z, w, scan_row(p, row, s.wsum[buf ^ 1]), s.wsum[buf ^ 1]);
    } else {
        const u64 at = place(p.u_sample[row], total);
        u64 before = 0;
        for (int c = 0; c < rank; ++c) before += s.total[buf][c];
        writes = at >= before && at < before + s.total[buf][rank];
        if (writes) {
            u64 r = at - before;
            int wi = 0;
            while (wi < kWarps - 1 && r >= s.wsum[buf][wi]) r -= s.wsum[buf][wi++];
            search(p, row, (rank * kWarps + wi) * p.sub, p.sub / 32, r, z, w, job.total, s.wsum[buf ^ 1],
                   [&](int v, const uint4 &x, u64 (&e)[kPer / 2]) { weights(x, drafts(v), e); });
        }
    }
    if (writes) row_done<1>(p);                                     // (a CTA of twice the warps)
}

template <bool kF32>
__global__ void __launch_bounds__(kThreads, 2) k_sample_draft(const SampleParams p)
{
    __shared__ Shared s;
    const cg::cluster_group cl = cg::this_cluster();
    const int C = (int)cl.num_blocks();
    pdl_wait();
    const int n = __ldcg(p.n_left);
    const int clusters = gridDim.x / C;
    cl.sync();                                                      // its CTAs have all started
    for (int i = blockIdx.x / C; i < n; i = s.next) {               // the same for the whole cluster
        const uint4 l = __ldcg(reinterpret_cast<const uint4 *>(p.left + i));
        reject<kF32>(p, s, cl, {(int32_t)l.x, __uint_as_float(l.y), (u64)l.w << 32 | l.z});
        cl.sync();                                                  // (they have all read the last one)
        if (cl.block_rank() == 0 && threadIdx.x < 32) {
            int next = threadIdx.x == 0 ? clusters + atomicAdd(p.taken, 1) : 0;
            next = __shfl_sync(0xffffffffu, next, 0);
            if (threadIdx.x < C) *cl.map_shared_rank(&s.next, threadIdx.x) = next;
        }
        cl.sync();
    }
}

}  // namespace

namespace w12i {

int64_t sample_max_vocab() { return kMaxVocab; }

static int64_t pieces_of(int64_t vocab, bool f32) { return (vocab + (f32 ? 4 : 8) - 1) / (f32 ? 4 : 8) + 1; }   // (a row may start inside one)

static int64_t chunk_count(int64_t vocab, bool f32, int per)
{
    return (pieces_of(vocab, f32) + kChunkThreads * per - 1) / (kChunkThreads * per);
}

// Pieces of a thread of the two passes: the most, of powers of two up to 16,
// that leave every SM eight CTAs.  Few rows are spread over the SMs; many get
// long stretches, over which a warp's sums and searches weigh less (256 FP32
// rows: the sums' pass takes 40 us with 16 pieces, 56 with 4).
static int pieces_per_thread(int64_t R, int64_t vocab, bool f32, int num_sms)
{
    int per = 16;
    while (per > 1 && R * chunk_count(vocab, f32, per) < 8ll * num_sms) per /= 2;
    return per;
}

template <bool kF32, int N>
static cudaError_t passes(cudaLaunchConfig_t &cfg, cudaLaunchAttribute *pdl, const SampleParams &p, bool draft)
{
    const cudaError_t e = cudaLaunchKernelEx(&cfg, k_sample_max<kF32, N>, p);
    if (e != cudaSuccess) return e;
    cfg.attrs = pdl;
    cfg.numAttrs = 1;
    return draft ? cudaLaunchKernelEx(&cfg, k_sample_sum<kF32, N, true>, p) : cudaLaunchKernelEx(&cfg, k_sample_sum<kF32, N, false>, p);
}

template <bool kF32>
static cudaError_t passes_of(cudaLaunchConfig_t &cfg, cudaLaunchAttribute *pdl, const SampleParams &p, bool draft)
{
    return p.per >= 4 ? passes<kF32, 4>(cfg, pdl, p, draft) : p.per == 2 ? passes<kF32, 2>(cfg, pdl, p, draft) : passes<kF32, 1>(cfg, pdl, p, draft);
}

static size_t align16(size_t x) { return (x + 15) & ~(size_t)15; }

// the counts, the rows left over, the maxima and the sums
size_t sample_scratch_bytes(int32_t R, int64_t vocab)
{
    const size_t chunks = (size_t)chunk_count(vocab, true, 1);
    return align16((size_t)(3 + R) * 4) + (size_t)R * sizeof(Left) + align16((size_t)R * chunks * 4) + (size_t)R * chunks * kChunkWarps * 8;
}

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
    p.status = a.status;
    p.per = pieces_per_thread(a.R, a.vocab, a.f32 != 0, a.num_sms);
    p.chunks = (int32_t)chunk_count(a.vocab, a.f32 != 0, p.per);
    uint8_t *scratch = static_cast<uint8_t *>(a.scratch);
    p.done = reinterpret_cast<int32_t *>(scratch);
    p.n_left = p.done + 1;
    p.taken = p.done + 2;
    p.arrived = p.done + 3;
    scratch += align16((size_t)(3 + a.R) * 4);
    p.left = reinterpret_cast<Left *>(scratch);
    scratch += (size_t)a.R * sizeof(Left);
    p.top = reinterpret_cast<float *>(scratch);
    p.sums = reinterpret_cast<u64 *>(scratch + align16((size_t)a.R * p.chunks * 4));
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)p.chunks, (unsigned)a.R);
    cfg.blockDim = dim3(kChunkThreads);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute pdl[1], both[2];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    const bool draft = a.draft_p != nullptr;
    const cudaError_t e = a.f32 ? passes_of<true>(cfg, pdl, p, draft) : passes_of<false>(cfg, pdl, p, draft);
    if (e != cudaSuccess || !draft) return (int)e;
    // A rejection's pass is one row's own, so a row gets all the CTAs a portable
    // cluster can have, down to 2048 tokens each.  (Clusters of 16: 256 rows in
    // 138 us against 121; fewer of them find room at a time.)
    int c = 1;
    while (c < kMaxCluster && a.vocab > 2048 * c) c *= 2;
    p.sub = (int32_t)((pieces_of(a.vocab, a.f32 != 0) + 32ll * c * kWarps - 1) / (32ll * c * kWarps) * 32);
    cfg.gridDim = dim3((unsigned)std::min(a.R * c, 2 * a.num_sms / c * c));
    cfg.blockDim = dim3(kThreads);
    both[0] = pdl[0];
    both[1].id = cudaLaunchAttributeClusterDimension;
    both[1].val.clusterDim.x = (unsigned)c;
    both[1].val.clusterDim.y = both[1].val.clusterDim.z = 1;
    cfg.attrs = both;
    cfg.numAttrs = 2;
    return (int)(a.f32 ? cudaLaunchKernelEx(&cfg, k_sample_draft<true>, p) : cudaLaunchKernelEx(&cfg, k_sample_draft<false>, p));
}

}  // namespace w12i
