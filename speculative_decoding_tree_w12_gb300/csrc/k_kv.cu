// Paged 8-bit KV cache: appending prompt rows and committing the accepted path
// of a draft tree, with the position rotation applied on the way.
//
// Mathematics.  A token's key is turned by its position (pairs (a, b) ->
// (a c - b s, b c + a s) in FP32, every product and sum rounded on its own, so
// a table and a position give one value whichever kernel computes it).  Keys
// and values are stored as E4M3 codes x / s under one power-of-two scale s per
// block of tokens and head: the least s with max|x| <= 448 s.  A block that
// already holds tokens keeps the larger of its scale and the new tokens'; its
// codes then move by a power of two, which is exact down to E4M3's subnormals.
// A power of two costs nothing against a finer scale (E4M3 is a floating
// format) and is what keeps a growing block from being rounded anew at every
// token.
//
// One CTA owns one block of tokens and a run of heads, so nothing is shared
// between CTAs but the lengths (see below).  It stages the positions' cosines and
// sines once; then for each head a warp takes consecutive tokens, a lane four
// dimensions, and what it works on stays in registers: rows, turned keys (a
// pair's other half comes from the lane that has it), the two maxima, codes (all
// 64 registers, and 48 to 56 bytes a thread spilled).  Keys
// leave token-major as they are; values are transposed through shared memory
// under an exclusive-or of the token group with the dimension, which keeps both
// sides free of most bank conflicts, and leave as whole rows of a dimension
// (the layout that the attention's V^T P product reads without a
// transposition).  What bounds a long prompt is memory, 4 bytes read and 2
// written for each pair of key and value elements, and next to it the issue of
// some 13 instructions an element between two barriers a head: 16 prompts of up
// to 8192 tokens with 8 heads (546 MB) take 123 us, 4.4 TB/s.  (Rows staged two
// heads ahead in shared memory took 20 us more.)
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "w12_device.cuh"
#include "w12_kv.cuh"

namespace {

using namespace w12d;
using namespace w12i;

struct KvParams {
    int32_t H, n_blocks, max_blocks, n_req, n_rows, heads;          // heads: of one CTA
    int64_t k_stride, v_stride;
    uint8_t *kc, *vc;
    float *ks, *vs;
    const int32_t *table, *len, *off;           // off: [n_req + 1] source rows of each request
    const int32_t *parent, *acc_node;           // commit: the path ending on acc_node[r]
    const uint16_t *k, *v;
    RopeArgs rope;
    int32_t *len_out, *arrive, *new_len, *status;
};

__device__ __forceinline__ void fail(int32_t *status) { atomicCAS(status, 0, (int32_t)W12_E_INVAL); }

__device__ __forceinline__ uint64_t pair(float a, float b)
{
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ uint64_t pair_bf16(uint32_t w) { return pair(bf16_lo(w), bf16_hi(w)); }
__device__ __forceinline__ float2 unpair(uint64_t d)
{
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(d));
    return f;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
// a b + c d, every operation rounded on its own: the sums one at a time, since
// a sum of two would be fused with a product of two before it
__device__ __forceinline__ uint64_t mul2_add2(uint64_t a, uint64_t b, uint64_t c, uint64_t d)
{
    const float2 x = unpair(mul2(a, b)), y = unpair(mul2(c, d));
    return pair(__fadd_rn(x.x, y.x), __fadd_rn(x.y, y.y));
}

// codes of two pairs of values, the first in the low byte.  `odd`: some may
// not be finite (their code is NaN, where the conversion alone would saturate).
__device__ __forceinline__ uint32_t codes4(uint64_t a, uint64_t b, bool odd)
{
    const float2 x = unpair(a), y = unpair(b);
    if (odd) return to_e4m3(x.x) | (to_e4m3(x.y) << 8) | (to_e4m3(y.x) << 16) | ((uint32_t)to_e4m3(y.y) << 24);
    return to_e4m3x2(x.x, x.y) | (to_e4m3x2(y.x, y.y) << 16);
}

// four codes under another scale
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float f)
{
    const float2 a = f16x2_f32(e4m3x2_f16x2(w & 0xFFFFu)), b = f16x2_f32(e4m3x2_f16x2(w >> 16));
    return to_e4m3x2(a.x * f, a.y * f) | (to_e4m3x2(b.x * f, b.y * f) << 16);
}

// the larger magnitude of a pair and t; `finite`: infinities count for nothing (a NaN never does)
__device__ __forceinline__ float top2(float t, uint64_t a, bool finite)
{
    const float2 x = unpair(a);
    if (!finite) return fmaxf(fmaxf(t, fabsf(x.x)), fabsf(x.y));
    if (fabsf(x.x) < INFINITY) t = fmaxf(t, fabsf(x.x));
    if (fabsf(x.y) < INFINITY) t = fmaxf(t, fabsf(x.y));
    return t;
}

// 1 / s of a power of two
__device__ __forceinline__ float inverse(float s) { return __uint_as_float((254u << 23) - __float_as_uint(s)); }

// words 0..3 of a 16-byte chunk in the order i ^ x
__device__ __forceinline__ uint4 xor_words(uint4 v, int x)
{
    if (x & 1) v = make_uint4(v.y, v.x, v.w, v.z);
    if (x & 2) v = make_uint4(v.z, v.w, v.x, v.y);
    return v;
}

// n tokens behind the length have their places in the table
__device__ __forceinline__ bool fits(const KvParams &p, int bt, int len, int n)
{
    return len >= 0 && (int64_t)len + n <= (int64_t)p.max_blocks * bt;
}

// BT: tokens of a block.  kCommit: the new tokens are the root path of
// acc_node[r], gathered by row; otherwise they are rows off[r] .. off[r + 1] - 1.
template <int BT, bool kCommit>
__global__ void __launch_bounds__(BT * 8, 128 / BT) k_kv_write(const KvParams p)
{
    constexpr int kTok = 4, kWarps = BT / kTok, kThreads = kWarps * 32;      // a warp takes four tokens
    extern __shared__ __align__(16) uint8_t smem[];
    uint8_t *tile = smem;                                            // [128][BT] value codes, token groups exchanged
    float *tab = reinterpret_cast<float *>(smem + BT * kKvDim);      // [tokens][rot / 2] cosines, then sines
    __shared__ int32_t s_path[kMaxDepth + 2];
    __shared__ int32_t s_parent[kMaxBudget];
    __shared__ int32_t s_r, s_item, s_n, s_ok;
    __shared__ uint2 s_top[kWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int h0 = blockIdx.y * p.heads, h1 = min(p.H, h0 + p.heads);

    // ---- which request and which of its blocks
    if (kCommit) {
        const int r = blockIdx.x;
        const int lo = p.off[r], hi = p.off[r + 1], end = p.acc_node[r];
        const bool in = lo >= 0 && hi <= p.n_rows && lo <= hi && (lo == hi || (end >= lo && end < hi));
        if (in && lo < hi)
            for (int j = lo + tid; j <= end; j += kThreads) s_parent[j - lo] = p.parent[j];
        __syncthreads();
        if (tid == 0) {
            int n = 0, ok = in;
            if (in && lo < hi) {
                int j = end;
                while (j >= lo && j <= end && n <= kMaxDepth + 1) {
                    s_path[n++] = j;
                    const int q = s_parent[j - lo];
                    if (q >= j) { ok = 0; break; }
                    j = q;
                }
                if (j >= 0 || n > kMaxDepth + 1) ok = 0;             // left the request, or too deep
            }
            s_r = r;
            s_item = blockIdx.z;
            s_n = ok ? n : 0;
            s_ok = ok;
        }
    } else if (warp == 0) {
        // items run over the requests' touched blocks in order
        int base = 0, found_r = -1, found_i = 0, found_n = 0, good = 1;
        int top = INT32_MIN;                                         // the largest offset so far, once one was out of order
        bool disorder = false;
        for (int r0 = 0; r0 < p.n_req && found_r < 0; r0 += 32) {
            const int r = r0 + lane;
            int n = 0, nb = 0, ok = 1, lo = 0, hi = 0, len = 0;
            if (r < p.n_req) lo = p.off[r], hi = p.off[r + 1], len = p.len[r];
            // the rows of the requests served lie one behind the other, so that the grid has a CTA for every block
            disorder |= __any_sync(0xffffffffu, lo > hi);
            if (disorder) {
                int m = r < p.n_req ? lo : INT32_MIN;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const int t = __shfl_up_sync(0xffffffffu, m, d);
                    if (lane >= d) m = max(m, t);
                }
                top = max(top, m);
                ok = lo >= top;
                top = __shfl_sync(0xffffffffu, top, 31);
            }
            if (r < p.n_req) {
                ok = ok && lo >= 0 && hi <= p.n_rows && lo <= hi && fits(p, BT, len, hi - lo);
                n = ok ? hi - lo : 0;
                nb = n ? (len + n - 1) / BT - len / BT + 1 : 1;      // a request without tokens still reports its length
            }
            int incl = nb;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int t = __shfl_up_sync(0xffffffffu, incl, d);
                if (lane >= d) incl += t;
            }
            const int x = (int)blockIdx.x - base;
            const unsigned in = __ballot_sync(0xffffffffu, r < p.n_req && x >= incl - nb && x < incl);
            if (in) {
                const int src = __ffs(in) - 1;
                found_r = r0 + src;
                found_i = x - (__shfl_sync(0xffffffffu, incl, src) - __shfl_sync(0xffffffffu, nb, src));
                found_n = __shfl_sync(0xffffffffu, n, src);
                good = __shfl_sync(0xffffffffu, ok, src);
            }
            base += __shfl_sync(0xffffffffu, incl, 31);
        }
        if (lane == 0) {
            s_r = found_r;
            s_item = found_i;
            s_n = found_n;
            s_ok = good;
        }
    }
    __syncthreads();
    const int r = s_r;
    const int item = s_item, len = r >= 0 ? p.len[r] : 0;
    const bool room = fits(p, BT, len, s_n);
    const int n_new = room ? s_n : 0;
    const int n_blk = n_new ? (len + n_new - 1) / BT - len / BT + 1 : 1;
    const bool has = r >= 0 && item < n_blk;                         // the grid is the largest that the rows can need
    bool ok = r >= 0 && s_ok && room && (p.rope.rot == 0 || n_new == 0 || len + n_new <= p.rope.max_pos);
    const int bi = len / BT + item;
    // every CTA of the request looks at all of its blocks, so that they agree
    const int32_t *table = p.table + (int64_t)max(r, 0) * p.max_blocks;
    int bad = 0;
    if (ok && n_new)
        for (int i = tid; i < n_blk; i += kThreads) {
            const int b = table[len / BT + i];
            bad |= b < 0 || b >= p.n_blocks;
        }
    if (__syncthreads_or(bad)) ok = false;
    const bool writes = ok && has && n_new;
    const int blk = writes ? table[bi] : 0;
    // ---- A length is written when every CTA that looks at it has done so: len_out
    // may be the cache's own array, and a CTA that has not started yet still
    // finds its block by it.  In an append that is any CTA of the grid, whose
    // last one writes all lengths (each request's first CTA leaves them in the
    // workspace); in a commit any CTA of the request.  So every CTA arrives,
    // those without a block too, and here, right behind its reads: the answer is
    // back by the time it is wanted (16 prompts of up to 8192 tokens: 123 us;
    // arriving at the end 126, and 133 with all warps waiting for the answer).
    int arrived = 0;
    if (tid == 0) {
        if (has && !ok) fail(p.status);
        if (!kCommit && has && item == 0 && blockIdx.y == 0) p.new_len[r] = ok ? len + n_new : len;
        __threadfence();
        arrived = atomicAdd(p.arrive + (kCommit ? r : 0), 1);
    }
    if (writes) {
        const int first = max(len, bi * BT);                         // positions [first, last) go into this block
        const int last = min(len + n_new, (bi + 1) * BT);
        const int held = first - bi * BT, end = last - bi * BT;      // slots it holds already; the new ones' end
        // ---- cosines and sines of the new positions
        const int half = p.rope.rot >> 1;
        float *sn = tab + BT * half;
        for (int i = tid; i < (end - held) * (half >> 2); i += kThreads) {
            reinterpret_cast<float4 *>(tab)[i] = __ldg(reinterpret_cast<const float4 *>(p.rope.cos + (int64_t)first * half) + i);
            reinterpret_cast<float4 *>(sn)[i] = __ldg(reinterpret_cast<const float4 *>(p.rope.sin + (int64_t)first * half) + i);
        }
        // this lane's four dimensions: what turns them, and where their partners are
        const int d0 = lane * 4;
        const bool turns = d0 < p.rope.rot, second = d0 >= half;
        const int f = p.rope.adjacent ? d0 >> 1 : second ? d0 - half : d0;
        const int mate = !turns || p.rope.adjacent ? lane : second ? lane - (half >> 2) : lane + (half >> 2);
        const int slot0 = warp * kTok;
        const int j0 = first - len - held + slot0;                   // the warp's first token's place among the request's new ones
        const int lo_i = max(held - slot0, 0), hi_i = min(end - slot0, kTok);   // of the warp's tokens, the new ones
        // each thread's 16-byte piece of the transposed values: dimension vd, tokens 16 vc ..
        const int vd = tid / (BT / 16), vc = tid % (BT / 16), vx = (vd >> 2) & (kWarps - 1);
        const uint4 *v_src = reinterpret_cast<const uint4 *>(tile + vd * BT) + (vc ^ (vx >> 2));
        uint32_t *v_tile = reinterpret_cast<uint32_t *>(tile + d0 * BT) + (warp ^ (lane & (kWarps - 1)));
        const float *tc = tab + (j0 - (first - len)) * half + f, *ts = tc + BT * half;
        const uint32_t flip = p.rope.adjacent || second ? 0u : 0x80008000u;    // a first half's partner counts negative
        int row[kTok];
#pragma unroll
        for (int i = 0; i < kTok; ++i) {
            const bool here = i >= lo_i && i < hi_i;
            row[i] = !here ? -1 : kCommit ? s_path[n_new - 1 - j0 - i] : p.off[r] + j0 + i;
        }
        __syncthreads();
        // kFull: every slot of the block is new, as in all of a long prompt but its ends
        auto heads = [&](auto full) {
            constexpr bool kFull = decltype(full)::value;
            uint2 kr[kTok], vr[kTok], vn[kTok];                      // next head's keys; this head's and the next one's values
            // the rows of head h; each is asked for as soon as the last head's are used up
            auto load = [&](uint2 (&x)[kTok], const uint16_t *src, int64_t stride, int h) {
                src += h * kKvDim + d0;
                if (kFull && !kCommit) {
                    src += row[0] * stride;
#pragma unroll
                    for (int i = 0; i < kTok; ++i, src += stride) x[i] = __ldg(reinterpret_cast<const uint2 *>(src));
                } else {
#pragma unroll
                    for (int i = 0; i < kTok; ++i) {
                        x[i] = make_uint2(0, 0);
                        if (row[i] >= 0) x[i] = __ldg(reinterpret_cast<const uint2 *>(src + row[i] * stride));
                    }
                }
            };
            load(kr, p.k, p.k_stride, h0);
            load(vn, p.v, p.v_stride, h0);
#pragma unroll 1
            for (int h = h0; h < h1; ++h) {
                const int64_t si = (int64_t)blk * p.H + h;
                const float k_old = held ? p.ks[si] : 0.f, v_old = held ? p.vs[si] : 0.f;
                // ---- turned keys, and the two maxima (of the values as they are: their bits order like their magnitudes)
#pragma unroll
                for (int i = 0; i < kTok; ++i) vr[i] = vn[i];
                uint64_t x[kTok][2];
                float tk = 0.f;
                uint32_t vm = 0;
#pragma unroll
                for (int i = 0; i < kTok; ++i) {
                    x[i][0] = pair_bf16(kr[i].x);
                    x[i][1] = pair_bf16(kr[i].y);
                    const uint32_t o0 = __shfl_sync(0xffffffffu, kr[i].x, mate) ^ flip, o1 = __shfl_sync(0xffffffffu, kr[i].y, mate) ^ flip;
                    if (turns && (kFull || row[i] >= 0)) {
                        uint64_t y[2], c[2], s[2];
                        if (p.rope.adjacent) {
                            const float2 cc = *reinterpret_cast<const float2 *>(tc + i * half), ss = *reinterpret_cast<const float2 *>(ts + i * half);
                            c[0] = pair(cc.x, cc.x), c[1] = pair(cc.y, cc.y);
                            s[0] = pair(-ss.x, ss.x), s[1] = pair(-ss.y, ss.y);
                            y[0] = pair(bf16_hi(kr[i].x), bf16_lo(kr[i].x));
                            y[1] = pair(bf16_hi(kr[i].y), bf16_lo(kr[i].y));
                        } else {
                            const float4 cc = *reinterpret_cast<const float4 *>(tc + i * half), ss = *reinterpret_cast<const float4 *>(ts + i * half);
                            c[0] = pair(cc.x, cc.y), c[1] = pair(cc.z, cc.w);
                            s[0] = pair(ss.x, ss.y), s[1] = pair(ss.z, ss.w);
                            y[0] = pair_bf16(o0), y[1] = pair_bf16(o1);
                        }
                        x[i][0] = mul2_add2(x[i][0], c[0], y[0], s[0]);
                        x[i][1] = mul2_add2(x[i][1], c[1], y[1], s[1]);
                    }
                    tk = top2(top2(tk, x[i][0], false), x[i][1], false);
                    vm = __vmaxu2(__vmaxu2(vm, vr[i].x & 0x7FFF7FFFu), vr[i].y & 0x7FFF7FFFu);
                }
                if (h + 1 < h1) {
                    load(kr, p.k, p.k_stride, h + 1);
                    load(vn, p.v, p.v_stride, h + 1);
                }
                float tv = __uint_as_float(max(vm & 0xFFFFu, vm >> 16) << 16);
                auto reduce = [&]() {                                    // over the CTA; magnitudes order like their bits
                    const uint32_t a = __reduce_max_sync(0xffffffffu, __float_as_uint(tk)), b = __reduce_max_sync(0xffffffffu, __float_as_uint(tv));
                    if (lane == 0) s_top[warp] = make_uint2(a, b);
                    __syncthreads();
                    const uint2 t = s_top[lane & (kWarps - 1)];
                    tk = __uint_as_float(__reduce_max_sync(0xffffffffu, t.x));
                    tv = __uint_as_float(__reduce_max_sync(0xffffffffu, t.y));
                };
                reduce();
                // an infinity (or, among the values, a NaN): count the finite values alone, convert with care
                const bool odd = !(tk < INFINITY) || !(tv < INFINITY);
                if (odd) {                                               // the same for the whole CTA
                    tk = tv = 0.f;
#pragma unroll
                    for (int i = 0; i < kTok; ++i) {
                        tk = top2(top2(tk, x[i][0], true), x[i][1], true);
                        tv = top2(top2(tv, pair_bf16(vr[i].x), true), pair_bf16(vr[i].y), true);
                    }
                    __syncthreads();
                    reduce();
                }
                float k_s = block_scale(tk), v_s = block_scale(tv);
                const bool k_re = held && k_s > k_old, v_re = held && v_s > v_old;
                if (held) k_s = fmaxf(k_s, k_old), v_s = fmaxf(v_s, v_old);
                const float k_i = inverse(k_s), v_i = inverse(v_s);
                const uint64_t k_i2 = pair(k_i, k_i), v_i2 = pair(v_i, v_i);
                uint8_t *gk = p.kc + si * (int64_t)(BT * kKvDim), *gv = p.vc + si * (int64_t)(BT * kKvDim);
                // ---- keys, and the held ones under a larger scale
                uint32_t *k_dst = reinterpret_cast<uint32_t *>(gk + slot0 * kKvDim) + lane;
                uint32_t vw[kTok];
#pragma unroll
                for (int i = 0; i < kTok; ++i) {
                    uint32_t *dst = k_dst + i * (kKvDim / 4);
                    if (kFull || row[i] >= 0) *dst = codes4(mul2(x[i][0], k_i2), mul2(x[i][1], k_i2), odd);
                    else if (k_re && slot0 + i < held) *dst = rescale4(*dst, k_old * k_i);
                    vw[i] = codes4(mul2(pair_bf16(vr[i].x), v_i2), mul2(pair_bf16(vr[i].y), v_i2), odd);
                }
                // ---- values: 4 dimensions x 4 tokens turned over, into the tile
                {
                    const uint32_t a = prmt(vw[0], vw[1], 0x5140u), b = prmt(vw[2], vw[3], 0x5140u);
                    const uint32_t c = prmt(vw[0], vw[1], 0x7362u), d = prmt(vw[2], vw[3], 0x7362u);
                    v_tile[0] = prmt(a, b, 0x5410u);
                    v_tile[BT / 4] = prmt(a, b, 0x7632u);
                    v_tile[2 * (BT / 4)] = prmt(c, d, 0x5410u);
                    v_tile[3 * (BT / 4)] = prmt(c, d, 0x7632u);
                }
                __syncthreads();
                uint4 w = xor_words(*v_src, vx & 3);
                uint4 *dst = reinterpret_cast<uint4 *>(gv) + tid;
                const int t = vc * 16;
                if (kFull) {
                    *dst = w;
                } else if (t + 16 > (v_re ? 0 : held) && t < end) {
                    if (t < held || t + 16 > end) {
                        // some of its tokens are old, or none yet: those bytes stay (or move to the larger scale)
                        const uint4 old = *dst;
                        uint32_t n[4] = {w.x, w.y, w.z, w.w}, q[4] = {old.x, old.y, old.z, old.w};
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int t4 = t + 4 * j;
                            const int a = min(max(held - t4, 0), 4), b = min(max(end - t4, 0), 4);   // new bytes a .. b - 1
                            const uint32_t below = a < 4 ? (1u << (8 * a)) - 1u : 0xFFFFFFFFu;
                            const uint32_t upto = b < 4 ? (1u << (8 * b)) - 1u : 0xFFFFFFFFu;
                            if (v_re) q[j] = bitmux(below, rescale4(q[j], v_old * v_i), q[j]);
                            n[j] = bitmux(upto & ~below, n[j], q[j]);
                        }
                        w = make_uint4(n[0], n[1], n[2], n[3]);
                    }
                    *dst = w;
                }
                if (tid == 0) {
                    p.ks[si] = k_s;
                    p.vs[si] = v_s;
                }
            }
        };
        if (held == 0 && end == BT) heads(std::true_type{});
        else heads(std::false_type{});
    }
    // ---- the last one writes the new lengths, and the counter goes back to zero for the next launch
    if (kCommit) {
        if (tid == 0 && arrived == (int)(gridDim.y * gridDim.z) - 1) {
            p.len_out[r] = ok ? len + n_new : len;
            p.arrive[r] = 0;
        }
        return;
    }
    if (warp) return;
    if (__shfl_sync(0xffffffffu, arrived, 0) != (int)(gridDim.x * gridDim.y) - 1) return;
    __threadfence();
    for (int i = lane; i < p.n_req; i += 32) p.len_out[i] = __ldcg(p.new_len + i);
    if (lane == 0) *p.arrive = 0;
}

}  // namespace

namespace w12i {

int launch_kv_write(const KvArgs &a, void *stream)
{
    KvParams p{};
    p.H = a.H;
    p.n_blocks = a.n_blocks;
    p.max_blocks = a.max_blocks;
    p.n_req = a.n_req;
    p.n_rows = a.n_rows;
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
    p.acc_node = a.acc_node;
    p.k = a.k;
    p.v = a.v;
    p.rope = a.rope;
    p.len_out = a.len_out;
    p.arrive = a.arrive;
    p.new_len = a.new_len;
    p.status = a.status;
    const bool commit = a.acc_node != nullptr;
    // blocks that one request's new tokens can touch: n tokens reach over at
    // most (n - 1) / bt + 2 of them.  A path's further blocks come last: most
    // of those CTAs have nothing to write (24 requests of 8 rows: 12.1 us with
    // a request's CTAs side by side)
    const unsigned items = commit ? kMaxDepth / a.bt + 2 : 1;
    const int64_t x = commit ? a.n_req : (int64_t)a.n_rows / a.bt + 2ll * a.n_req;
    // Heads of a CTA: so many that all touched blocks' CTAs fit the SMs at once
    // (128 / bt of them an SM), since a CTA spends some 4 us on finding its
    // block and staging the tables before its first head, and a head's loads
    // hide behind the head before.  24 prompts of 700 tokens at most, blocks of
    // 32: all 4 heads to a CTA 16.4 us, one 18.4; 16 of up to 8192 tokens: all
    // 8 heads 123 us, 4 of them 133, one 229; 24 paths of a tree of 192 rows with
    // 8 heads: one 13 to 16 us, all 8 21.
    const int64_t blocks = (commit ? 0 : (int64_t)a.n_rows / a.bt) + a.n_req;
    const int64_t parts = std::min<int64_t>(a.H, std::max<int64_t>(1, 128 / a.bt * a.num_sms / blocks));
    p.heads = (int32_t)((a.H + parts - 1) / parts);
    const dim3 grid((unsigned)x, (unsigned)((a.H + p.heads - 1) / p.heads), items);
    const int smem = a.bt * (kKvDim + a.rope.rot * 4);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaSuccess;
    auto go = [&](auto kernel, int threads) {
        // (static shared memory counts too: up to 2.4 KB)
        if (smem > 44 * 1024) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return;
        kernel<<<grid, threads, smem, st>>>(p);
        e = cudaGetLastError();
    };
    if (a.bt == 32) commit ? go(k_kv_write<32, true>, 256) : go(k_kv_write<32, false>, 256);
    else if (a.bt == 64) commit ? go(k_kv_write<64, true>, 512) : go(k_kv_write<64, false>, 512);
    else commit ? go(k_kv_write<128, true>, 1024) : go(k_kv_write<128, false>, 1024);
    return (int)e;
}

}  // namespace w12i
