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
// One CTA owns one block of one head, so nothing is shared between CTAs but
// the lengths (below).  It stages the block's new rows in shared memory, takes
// the two maxima, and writes the codes: keys token-major, values transposed
// (the layout the attention's P.V product reads without a transposition).
#include <cuda_runtime.h>

#include <cstdint>

#include "w12_device.cuh"
#include "w12_kv.cuh"

namespace {

using namespace w12d;
using namespace w12i;

constexpr int kThreads = 256;
constexpr int kPad = 8;                         // bf16 per staged row, against bank conflicts
constexpr int kRow = kKvDim + kPad;

struct KvParams {
    int32_t H, bt, n_blocks, max_blocks, n_req, n_rows, items;
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

// kCommit: the new tokens are the root path of acc_node[r], gathered by row;
// otherwise they are rows off[r] .. off[r + 1] - 1.
template <bool kCommit>
__global__ void __launch_bounds__(kThreads) k_kv_write(const KvParams p)
{
    extern __shared__ __align__(16) uint8_t smem[];
    uint16_t *sk = reinterpret_cast<uint16_t *>(smem);              // [bt][kRow] source rows (BF16 bits)
    uint16_t *sv = sk + p.bt * kRow;
    uint8_t *ck = reinterpret_cast<uint8_t *>(sv + p.bt * kRow);    // [bt][128] key codes
    uint8_t *cv = ck + p.bt * kKvDim;                               // [128][bt] value codes
    __shared__ int32_t s_path[kMaxDepth + 2];
    __shared__ int32_t s_r, s_item, s_n, s_ok;
    __shared__ float s_top[2][kThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int h = blockIdx.y;

    // ---- which request and which of its blocks
    if (kCommit) {
        if (warp == 0) {
            const int r = blockIdx.x / p.items;
            const int lo = p.off[r], hi = p.off[r + 1];
            int n = 0, ok = 1;
            if (lane == 0) {
                if (lo < 0 || hi > p.n_rows || lo > hi) ok = 0;
                int j = p.acc_node[r];
                if (ok && lo < hi) {
                    while (j >= lo && j < hi && n <= kMaxDepth + 1) {
                        s_path[n++] = j;
                        const int q = p.parent[j];
                        if (q >= j) { ok = 0; break; }
                        j = q;
                    }
                    if (j >= 0 || n > kMaxDepth + 1 || n == 0) ok = 0;   // left the request, or too deep
                }
                s_r = r;
                s_item = blockIdx.x % p.items;
                s_n = ok ? n : 0;
                s_ok = ok;
            }
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
                nb = n ? (len + n - 1) / p.bt - len / p.bt + 1 : 1;      // a request without tokens still reports its length
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
    const int n_new = s_n;
    const int len = p.len[r];
    const int bt = p.bt;
    const int n_blk = n_new ? (len + n_new - 1) / bt - len / bt + 1 : 1;
    const int item = s_item;
    if (item >= n_blk) return;
    bool ok = s_ok && len >= 0 && (int64_t)len + n_new <= (int64_t)p.max_blocks * bt &&
              (p.rope.rot == 0 || n_new == 0 || len + n_new <= p.rope.max_pos);
    const int bi = len / bt + item;
    // every CTA of the request looks at all of its blocks, so that they agree
    const int32_t *table = p.table + (int64_t)r * p.max_blocks;
    int bad = 0;
    if (ok && n_new)
        for (int i = tid; i < n_blk; i += kThreads) {
            const int b = table[len / bt + i];
            bad |= b < 0 || b >= p.n_blocks;
        }
    if (__syncthreads_or(bad)) ok = false;
    const int blk = ok && n_new ? table[bi] : 0;
    if (!ok && tid == 0) fail(p.status);
    if (ok && n_new) {
        const int first = max(len, bi * bt);                      // positions [first, last) go into this block
        const int last = min(len + n_new, (bi + 1) * bt);
        const int slot0 = first - bi * bt, cnt = last - first;
        const int held = slot0;                                    // tokens that the block holds already
        // ---- stage the source rows
        for (int i = tid; i < cnt * 16; i += kThreads) {
            const int t = i >> 4, c = (i & 15) * 8;
            const int j = first - len + t;
            const int64_t row = kCommit ? s_path[n_new - 1 - j] : p.off[r] + j;
            *reinterpret_cast<uint4 *>(sk + t * kRow + c) =
                __ldg(reinterpret_cast<const uint4 *>(p.k + row * p.k_stride + (int64_t)h * kKvDim + c));
            *reinterpret_cast<uint4 *>(sv + t * kRow + c) =
                __ldg(reinterpret_cast<const uint4 *>(p.v + row * p.v_stride + (int64_t)h * kKvDim + c));
        }
        __syncthreads();
        // ---- the two maxima over finite values
        float tk = 0.f, tv = 0.f;
        for (int i = tid; i < cnt * kKvDim; i += kThreads) {
            const int t = i / kKvDim, d = i % kKvDim;
            const float x = fabsf(rotated(sk + t * kRow, d, first + t, p.rope));
            const float y = fabsf(bf16_f32(sv[t * kRow + d]));
            if (x < INFINITY) tk = fmaxf(tk, x);
            if (y < INFINITY) tv = fmaxf(tv, y);
        }
#pragma unroll
        for (int d = 16; d; d >>= 1) {
            tk = fmaxf(tk, __shfl_xor_sync(0xffffffffu, tk, d));
            tv = fmaxf(tv, __shfl_xor_sync(0xffffffffu, tv, d));
        }
        if (lane == 0) s_top[0][warp] = tk, s_top[1][warp] = tv;
        __syncthreads();
        tk = tv = 0.f;
        for (int w = 0; w < kThreads / 32; ++w) tk = fmaxf(tk, s_top[0][w]), tv = fmaxf(tv, s_top[1][w]);
        const int64_t si = (int64_t)blk * p.H + h;
        float k_s = block_scale(tk), v_s = block_scale(tv);
        const float k_old = p.ks[si], v_old = p.vs[si];
        bool k_re = false, v_re = false;
        if (held) {
            k_re = k_s > k_old;
            v_re = v_s > v_old;
            k_s = fmaxf(k_s, k_old);
            v_s = fmaxf(v_s, v_old);
        }
        uint8_t *gk = p.kc + si * (int64_t)(bt * kKvDim), *gv = p.vc + si * (int64_t)(bt * kKvDim);
        // ---- codes of the tokens held already, under the larger scale
        if (k_re)
            for (int i = tid; i < held * kKvDim; i += kThreads) ck[i] = to_e4m3(e4m3_f32(gk[i]) * (k_old / k_s));
        if (v_re)
            for (int i = tid; i < held * kKvDim; i += kThreads) {
                const int d = i / held, t = i % held;
                cv[d * bt + t] = to_e4m3(e4m3_f32(gv[d * bt + t]) * (v_old / v_s));
            }
        // ---- codes of the new ones
        const float k_i = 1.f / k_s, v_i = 1.f / v_s;              // exact: powers of two
        for (int i = tid; i < cnt * kKvDim; i += kThreads) {
            const int t = i / kKvDim, d = i % kKvDim;
            ck[(slot0 + t) * kKvDim + d] = to_e4m3(rotated(sk + t * kRow, d, first + t, p.rope) * k_i);
            cv[d * bt + slot0 + t] = to_e4m3(bf16_f32(sv[t * kRow + d]) * v_i);
        }
        __syncthreads();
        // ---- write the slots that changed
        const int wk = k_re ? 0 : slot0, wv = v_re ? 0 : slot0, we = slot0 + cnt;
        for (int i = tid; i < (we - wk) * 8; i += kThreads)
            reinterpret_cast<uint4 *>(gk)[wk * 8 + i] = reinterpret_cast<uint4 *>(ck)[wk * 8 + i];
        if (wv == 0 && we == bt) {
            for (int i = tid; i < bt * 8; i += kThreads)
                reinterpret_cast<uint4 *>(gv)[i] = reinterpret_cast<uint4 *>(cv)[i];
        } else {
            const int w = we - wv;
            for (int i = tid; i < w * kKvDim; i += kThreads) {
                const int d = i / w, t = wv + i % w;
                gv[d * bt + t] = cv[d * bt + t];
            }
        }
        if (tid == 0) {
            p.ks[si] = k_s;
            p.vs[si] = v_s;
        }
    }
    // ---- the request's last CTA to get here writes its length (len_out may be
    // the cache's own array: every CTA has read it by then).  The counter goes
    // back to zero for the next launch.
    __syncthreads();
    if (tid == 0) {
        const int total = n_blk * p.H;
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
    p.bt = a.bt;
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
    const int smem = a.bt * (2 * kRow * 2 + 2 * kKvDim);
    const bool commit = a.acc_node != nullptr;
    // blocks that one request's new tokens can touch: n tokens reach over at
    // most (n - 1) / bt + 2 of them
    p.items = kMaxDepth / a.bt + 2;
    const int64_t x = commit ? (int64_t)a.n_req * p.items : (int64_t)a.n_rows / a.bt + 2ll * a.n_req;
    const dim3 grid((unsigned)x, (unsigned)a.H);
    const void *f = commit ? (const void *)k_kv_write<true> : (const void *)k_kv_write<false>;
    cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return (int)e;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (commit)
        k_kv_write<true><<<grid, kThreads, smem, st>>>(p);
    else
        k_kv_write<false><<<grid, kThreads, smem, st>>>(p);
    return (int)cudaGetLastError();
}

}  // namespace w12i
