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
// between CTAs but the lengths (below).  It stages the positions' cosines and
// sines once; then for each head a warp takes consecutive tokens, a lane four
// dimensions, and everything stays in registers: rows, turned keys (a pair's
// other half comes from the lane that has it), the two maxima, codes.  Keys
// leave token-major as they are; values are transposed through shared memory
// under an exclusive-or of the token group with the dimension, which keeps both
// sides free of most bank conflicts, and leave as whole rows of a dimension
// (the layout that the attention's V^T P product reads without a
// transposition).  What bounds a long prompt is memory: 4 bytes read and 2
// written for each pair of key and value elements.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "w12_device.cuh"
#include "w12_kv.cuh"

namespace {

using namespace w12d;
using namespace w12i;

struct KvParams {
    int32_t H, n_blocks, max_blocks, n_req, n_rows, items, heads;   // heads: of one CTA
    int64_t k_stride, v_stride;
    uint8_t *kc, *vc;
    float *ks, *vs;
    const int32_t *table, *len, *off;           // off: [n_req + 1] source rows of each request
    const int32_t *parent, *acc_node;           // commit: the path ending on acc_node[r]
    const uint16_t *k, *v;
    RopeArgs rope;
    int32_t *len_out, *arrive, *status;
};

__device__ __forceinline__ void fail(int32_t *status) { atomicCAS(status, 0, (int32_t)W12_E_INVAL); }

// codes of four values (not finite: NaN), the first in the low byte
__device__ __forceinline__ uint32_t codes4(float4 x)
{
    if (!(fmaxf(fmaxf(fabsf(x.x), fabsf(x.y)), fmaxf(fabsf(x.z), fabsf(x.w))) <= 448.f))
        return to_e4m3(x.x) | (to_e4m3(x.y) << 8) | (to_e4m3(x.z) << 16) | ((uint32_t)to_e4m3(x.w) << 24);
    return to_e4m3x2(x.x, x.y) | (to_e4m3x2(x.z, x.w) << 16);
}

// four codes under another scale
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float f)
{
    const float2 a = f16x2_f32(e4m3x2_f16x2(w & 0xFFFFu)), b = f16x2_f32(e4m3x2_f16x2(w >> 16));
    return to_e4m3x2(a.x * f, a.y * f) | (to_e4m3x2(b.x * f, b.y * f) << 16);
}

__device__ __forceinline__ float top4(float t, float4 x)
{
    const float a[4] = {fabsf(x.x), fabsf(x.y), fabsf(x.z), fabsf(x.w)};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (a[i] < INFINITY) t = fmaxf(t, a[i]);
    return t;
}

// words 0..3 of a 16-byte chunk in the order i ^ x
__device__ __forceinline__ uint4 xor_words(uint4 v, int x)
{
    if (x & 1) v = make_uint4(v.y, v.x, v.w, v.z);
    if (x & 2) v = make_uint4(v.z, v.w, v.x, v.y);
    return v;
}

// BT: tokens of a block.  kCommit: the new tokens are the root path of
// acc_node[r], gathered by row; otherwise they are rows off[r] .. off[r + 1] - 1.
template <int BT, bool kCommit>
__global__ void __launch_bounds__(BT == 32 ? 256 : 512, 2) k_kv_write(const KvParams p)
{
    constexpr int kWarps = BT == 32 ? 8 : 16, kThreads = kWarps * 32, kTok = BT / kWarps;   // tokens of a warp: 4 or 8
    extern __shared__ __align__(16) uint8_t smem[];
    uint8_t *tile = smem;                                            // [128][BT] value codes, token groups exchanged
    float *tab = reinterpret_cast<float *>(smem + BT * kKvDim);      // [tokens][rot / 2] cosines, then sines
    __shared__ int32_t s_path[kMaxDepth + 2];
    __shared__ int32_t s_parent[kMaxBudget];
    __shared__ int32_t s_r, s_item, s_n, s_ok;
    __shared__ float s_top[2][kWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int h0 = blockIdx.y * p.heads, h1 = min(p.H, h0 + p.heads);

    // ---- which request and which of its blocks
    if (kCommit) {
        const int r = blockIdx.x / p.items;
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
            s_item = blockIdx.x % p.items;
            s_n = ok ? n : 0;
            s_ok = ok;
        }
    } else if (warp == 0) {
        // items run over the requests' touched blocks in order
        int base = 0, found_r = -1, found_i = 0, found_n = 0, good = 1;
        for (int r0 = 0; r0 < p.n_req && found_r < 0; r0 += 32) {
            const int r = r0 + lane;
            int n = 0, nb = 0, ok = 1;
            if (r < p.n_req) {
                const int lo = p.off[r], hi = p.off[r + 1], len = p.len[r];
                ok = lo >= 0 && hi <= p.n_rows && lo <= hi && len >= 0;
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
    if (r < 0) return;
    const int n_new = s_n, item = s_item, len = p.len[r];
    const int n_blk = n_new ? (len + n_new - 1) / BT - len / BT + 1 : 1;
    if (item >= n_blk) return;
    bool ok = s_ok && len >= 0 && (int64_t)len + n_new <= (int64_t)p.max_blocks * BT &&
              (p.rope.rot == 0 || n_new == 0 || len + n_new <= p.rope.max_pos);
    const int bi = len / BT + item;
    // every CTA of the request looks at all of its blocks, so that they agree
    const int32_t *table = p.table + (int64_t)r * p.max_blocks;
    int bad = 0;
    if (ok && n_new)
        for (int i = tid; i < n_blk; i += kThreads) {
            const int b = table[len / BT + i];
            bad |= b < 0 || b >= p.n_blocks;
        }
    if (__syncthreads_or(bad)) ok = false;
    const int blk = ok && n_new ? table[bi] : 0;
    if (!ok && tid == 0) fail(p.status);
    if (ok && n_new) {
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
        const int64_t row0 = kCommit ? 0 : p.off[r] + (int64_t)(first - len) - held;
        __syncthreads();
#pragma unroll 1
        for (int h = h0; h < h1; ++h) {
            const int64_t si = (int64_t)blk * p.H + h;
            const float k_old = p.ks[si], v_old = p.vs[si];
            uint2 kr[kTok], vr[kTok];
#pragma unroll
            for (int i = 0; i < kTok; ++i) {
                const int slot = slot0 + i;
                kr[i] = vr[i] = make_uint2(0, 0);
                if (slot >= held && slot < end) {
                    const int64_t row = kCommit ? (int64_t)s_path[n_new - 1 - (first - len) - (slot - held)] : row0 + slot;
                    kr[i] = __ldg(reinterpret_cast<const uint2 *>(p.k + row * p.k_stride + (int64_t)h * kKvDim + d0));
                    vr[i] = __ldg(reinterpret_cast<const uint2 *>(p.v + row * p.v_stride + (int64_t)h * kKvDim + d0));
                }
            }
            // ---- turned keys, and the two maxima over finite values
            float4 x[kTok];
            float tk = 0.f, tv = 0.f;
#pragma unroll
            for (int i = 0; i < kTok; ++i) {
                const int slot = slot0 + i;
                x[i] = make_float4(bf16_lo(kr[i].x), bf16_hi(kr[i].x), bf16_lo(kr[i].y), bf16_hi(kr[i].y));
                const uint2 o = make_uint2(__shfl_sync(0xffffffffu, kr[i].x, mate), __shfl_sync(0xffffffffu, kr[i].y, mate));
                if (turns && slot >= held && slot < end) {
                    float4 c, s, y;
                    if (p.rope.adjacent) {
                        const float2 cc = *reinterpret_cast<const float2 *>(tab + (slot - held) * half + f);
                        const float2 ss = *reinterpret_cast<const float2 *>(sn + (slot - held) * half + f);
                        c = make_float4(cc.x, cc.x, cc.y, cc.y);
                        s = make_float4(-ss.x, ss.x, -ss.y, ss.y);
                        y = make_float4(x[i].y, x[i].x, x[i].w, x[i].z);
                    } else {
                        c = *reinterpret_cast<const float4 *>(tab + (slot - held) * half + f);
                        s = *reinterpret_cast<const float4 *>(sn + (slot - held) * half + f);
                        if (!second) s = make_float4(-s.x, -s.y, -s.z, -s.w);
                        y = make_float4(bf16_lo(o.x), bf16_hi(o.x), bf16_lo(o.y), bf16_hi(o.y));
                    }
                    x[i] = make_float4(__fadd_rn(__fmul_rn(x[i].x, c.x), __fmul_rn(y.x, s.x)),
                                       __fadd_rn(__fmul_rn(x[i].y, c.y), __fmul_rn(y.y, s.y)),
                                       __fadd_rn(__fmul_rn(x[i].z, c.z), __fmul_rn(y.z, s.z)),
                                       __fadd_rn(__fmul_rn(x[i].w, c.w), __fmul_rn(y.w, s.w)));
                }
                tk = top4(tk, x[i]);
                tv = top4(tv, make_float4(bf16_lo(vr[i].x), bf16_hi(vr[i].x), bf16_lo(vr[i].y), bf16_hi(vr[i].y)));
            }
#pragma unroll
            for (int d = 16; d; d >>= 1) {
                tk = fmaxf(tk, __shfl_xor_sync(0xffffffffu, tk, d));
                tv = fmaxf(tv, __shfl_xor_sync(0xffffffffu, tv, d));
            }
            if (lane == 0) s_top[0][warp] = tk, s_top[1][warp] = tv;
            __syncthreads();
            tk = tv = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) tk = fmaxf(tk, s_top[0][w]), tv = fmaxf(tv, s_top[1][w]);
            float k_s = block_scale(tk), v_s = block_scale(tv);
            bool k_re = false, v_re = false;
            if (held) {
                k_re = k_s > k_old;
                v_re = v_s > v_old;
                k_s = fmaxf(k_s, k_old);
                v_s = fmaxf(v_s, v_old);
            }
            const float k_i = 1.f / k_s, v_i = 1.f / v_s;            // exact: powers of two
            uint8_t *gk = p.kc + si * (int64_t)(BT * kKvDim), *gv = p.vc + si * (int64_t)(BT * kKvDim);
            // ---- keys, and the held ones under a larger scale
            uint32_t vw[kTok];
#pragma unroll
            for (int i = 0; i < kTok; ++i) {
                const int slot = slot0 + i;
                uint32_t *dst = reinterpret_cast<uint32_t *>(gk + slot * kKvDim) + lane;
                if (slot >= held && slot < end)
                    *dst = codes4(make_float4(x[i].x * k_i, x[i].y * k_i, x[i].z * k_i, x[i].w * k_i));
                else if (slot < held && k_re)
                    *dst = rescale4(*dst, k_old / k_s);
                vw[i] = codes4(make_float4(bf16_lo(vr[i].x) * v_i, bf16_hi(vr[i].x) * v_i, bf16_lo(vr[i].y) * v_i,
                                           bf16_hi(vr[i].y) * v_i));
            }
            // ---- values: 4 dimensions x 4 tokens at a time turned over, into the tile
#pragma unroll
            for (int i = 0; i < kTok; i += 4) {
                const uint32_t a = prmt(vw[i], vw[i + 1], 0x5140u), b = prmt(vw[i + 2], vw[i + 3], 0x5140u);
                const uint32_t c = prmt(vw[i], vw[i + 1], 0x7362u), d = prmt(vw[i + 2], vw[i + 3], 0x7362u);
                vw[i] = prmt(a, b, 0x5410u);
                vw[i + 1] = prmt(a, b, 0x7632u);
                vw[i + 2] = prmt(c, d, 0x5410u);
                vw[i + 3] = prmt(c, d, 0x7632u);
            }
            const int group = warp ^ (lane & (kWarps - 1));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint8_t *dst = tile + (d0 + i) * BT + group * kTok;
                if (kTok == 8) *reinterpret_cast<uint2 *>(dst) = make_uint2(vw[i], vw[i + 4 < kTok ? i + 4 : i]);
                else *reinterpret_cast<uint32_t *>(dst) = vw[i];
            }
            __syncthreads();
            for (int i = tid; i < BT * kKvDim / 16; i += kThreads) {
                const int d = i / (BT / 16), c = i % (BT / 16), x4 = (d >> 2) & (kWarps - 1);
                const int t = c * 16;
                if (t + 16 <= (v_re ? 0 : held) || t >= end) continue;               // nothing here changes
                uint4 w;
                if (kTok == 8) {
                    w = *reinterpret_cast<const uint4 *>(tile + d * BT + ((2 * c) ^ (x4 & ~1)) * 8);
                    if (x4 & 1) w = make_uint4(w.z, w.w, w.x, w.y);
                } else {
                    w = xor_words(*reinterpret_cast<const uint4 *>(tile + d * BT + (c ^ (x4 >> 2)) * 16), x4 & 3);
                }
                uint4 *dst = reinterpret_cast<uint4 *>(gv + d * BT) + c;
                if (t < held || t + 16 > end) {
                    // some of its tokens are old, or none yet: those bytes stay (or move to the larger scale)
                    uint4 old = *dst;
                    uint32_t n[4] = {w.x, w.y, w.z, w.w}, q[4] = {old.x, old.y, old.z, old.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int t4 = t + 4 * j;
                        const int a = min(max(held - t4, 0), 4), b = min(max(end - t4, 0), 4);   // new bytes a .. b - 1
                        const uint32_t below = a < 4 ? (1u << (8 * a)) - 1u : 0xFFFFFFFFu;
                        const uint32_t upto = b < 4 ? (1u << (8 * b)) - 1u : 0xFFFFFFFFu;
                        if (v_re) q[j] = bitmux(below, rescale4(q[j], v_old / v_s), q[j]);
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
    }
    // ---- the request's last CTA to get here writes its length (len_out may be
    // the cache's own array: every CTA has read it by then).  The counter goes
    // back to zero for the next launch.
    __syncthreads();
    if (tid == 0) {
        const int total = n_blk * (int)gridDim.y;
        __threadfence();
        if (atomicAdd(p.arrive + r, 1) == total - 1) {
            p.arrive[r] = 0;
            p.len_out[r] = ok ? len + n_new : len;
        }
    }
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
    p.status = a.status;
    // Heads of a CTA: as many as leave two CTAs to an SM (each one more shares
    // the staged tables; fewer spread a short prompt)
    const bool commit = a.acc_node != nullptr;
    // blocks that one request's new tokens can touch: n tokens reach over at
    // most (n - 1) / bt + 2 of them
    p.items = kMaxDepth / a.bt + 2;
    const int64_t x = commit ? (int64_t)a.n_req * p.items : (int64_t)a.n_rows / a.bt + 2ll * a.n_req;
    const int64_t blocks = commit ? a.n_req : std::max<int64_t>(a.n_rows / a.bt, 1);
    p.heads = (int32_t)std::min<int64_t>(a.H, std::max<int64_t>(1, blocks * a.H / (2 * a.num_sms)));
    const dim3 grid((unsigned)x, (unsigned)((a.H + p.heads - 1) / p.heads));
    const int smem = a.bt * (kKvDim + a.rope.rot * 4);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaSuccess;
    auto go = [&](auto kernel, int threads) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return;
        kernel<<<grid, threads, smem, st>>>(p);
        e = cudaGetLastError();
    };
    if (a.bt == 32) commit ? go(k_kv_write<32, true>, 256) : go(k_kv_write<32, false>, 256);
    else if (a.bt == 64) commit ? go(k_kv_write<64, true>, 512) : go(k_kv_write<64, false>, 512);
    else commit ? go(k_kv_write<128, true>, 512) : go(k_kv_write<128, false>, 512);
    return (int)e;
}

}  // namespace w12i
