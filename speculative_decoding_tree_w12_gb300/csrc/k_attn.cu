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
// k_attn_ctx: the cached context.  The work is a list of tiles of 128 tokens
// (request, key/value head, group of rows; tokens innermost), cut into equal
// consecutive shares, one per CTA and one CTA per SM, so a long context of one
// request and many short ones balance alike.  A share leaves, for every
// segment (request, head, group) that it meets, FP32 sums with their maximum
// and normaliser; k_attn_join merges them with the root path's.
//
// Tokens lie on the 128 lanes of tensor memory, query rows (rows x heads of
// the group, padded to 16) on its columns: few queries cost few columns, not
// an empty 128-row tile, and the cached codes are the A operand of both
// products, which is read once per tile whatever the number of queries.
//   S^T = K Q^T  kind::f8f6f4: K's codes as they lie in the cache; Q in three
//                E4M3 pieces that add up to twelve significant bits (2^-17 of
//                the head's largest at least), one product each into the same
//                accumulators.
//   O^T = V^T P  kind::f16: V's codes widened to F16 (exact) by a warpgroup of
//                its own; P in F16, eleven significant bits, scaled so that
//                there are 2^-18 below a weight of 1 before the subnormals.
// The maximum is lazy: P refers to a column maximum that is only raised when a
// score passes it by 2^6 (P stays under F16's top), so the usual tile has no
// reduction over lanes at all; the same slow path raises the reference of the
// value scales, which P carries.
#include <cuda.h>
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
constexpr int kCols = 80;                  // query rows of a segment: shared memory holds three Q pieces and two P tiles of them
constexpr int kTile = 128;                 // tokens of a tile
constexpr int kStages = 3;                 // K and V tiles in flight
constexpr int kScaleRing = 8;              // tiles whose block scales are kept (the producer runs at most 4 ahead of their readers)
constexpr int kMaxReq = kMaxBudget;
constexpr int kThreads = 512;              // warps: 0 producer, 1 MMA, 4-11 softmax, 12-15 V conversion
constexpr int kSoft = 256;
constexpr int kChunks = 3;                 // 16-column chunks of one softmax warpgroup (of kCols / 16 in all)
constexpr float kHead = 16.f;              // P of a weight of 1 under the reference scale
constexpr float kRaise = 6.f;              // a score may pass the column's reference by this (log2) before it is raised
constexpr float kScaleRaise = 16.f;        // ... and a value scale its reference by this factor: 16 * 2^6 * 16 < 2^15

struct AttnParams {
    int32_t H, Hq, G, bt, n_blocks, max_blocks, n_req, R, ctas;
    int64_t q_stride, k_stride, v_stride;
    const uint8_t *kc, *vc;
    const float *ks, *vs;
    const int32_t *table, *len, *off, *parent, *req;
    const uint8_t *depth;
    const uint16_t *q, *k, *v;
    RopeArgs rope;
    float scale2;                           // softmax scale * log2(e)
    uint16_t *out;
    int64_t *plan;                          // [n_req + 1] first tile of every request
    float *part;                            // [R * Hq + ctas * kCols][kD] sums
    float2 *ml;                             // [R * Hq + ctas * kCols] maximum (log2), normaliser
    int32_t *status;
    uint64_t timeout_ns;
};

__device__ __forceinline__ void fail(int32_t *status) { atomicCAS(status, 0, (int32_t)W12_E_INVAL); }

// rows of a request's groups: as many as fit the columns, evenly
__host__ __device__ __forceinline__ int group_count(int rows, int G) { return (rows + kCols / G - 1) / (kCols / G); }
__device__ __forceinline__ int group_rows(int rows, int G)
{
    const int g = group_count(rows, G);
    return (rows + g - 1) / g;
}

// a request's rows and cached tokens; false where they contradict each other or the tables
__device__ __forceinline__ bool request_ok(const AttnParams &p, int r, int &lo, int &rows, int &len)
{
    lo = p.off[r];
    const int hi = p.off[r + 1];
    len = p.len[r];
    rows = hi - lo;
    return lo >= 0 && hi <= p.R && rows >= 0 && len >= 0 && (int64_t)len <= (int64_t)p.max_blocks * p.bt;
}

// the request of a row, or -1
__device__ __forceinline__ int request_of(const AttnParams &p, int row)
{
    const int r = p.req[row];
    if (r < 0 || r >= p.n_req) return -1;
    int lo, rows, len;
    if (!request_ok(p, r, lo, rows, len) || row < lo || row >= lo + rows) return -1;
    if (p.rope.rot && len + (int)p.depth[row] >= p.rope.max_pos) return -1;
    return r;
}

// four consecutive elements d0 .. d0 + 3 of a BF16 row, turned by position pos
__device__ __forceinline__ void rotated4(const uint16_t *row, int d0, int pos, const RopeArgs &r, float (&x)[4])
{
    const uint2 w = __ldg(reinterpret_cast<const uint2 *>(row + d0));
    x[0] = bf16_f32((uint16_t)w.x);
    x[1] = bf16_f32((uint16_t)(w.x >> 16));
    x[2] = bf16_f32((uint16_t)w.y);
    x[3] = bf16_f32((uint16_t)(w.y >> 16));
    if (d0 >= r.rot) return;
    if (r.rot & 7) {                        // pairs that cross the groups of four
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = rotated(row, d0 + i, pos, r);
        return;
    }
    const int half = r.rot >> 1;
    const float *ct = r.cos + (int64_t)pos * half, *st = r.sin + (int64_t)pos * half;
    if (r.adjacent) {
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
            const float c = __ldg(ct + ((d0 + i) >> 1)), s = __ldg(st + ((d0 + i) >> 1));
            const float a = x[i], b = x[i + 1];
            x[i] = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
            x[i + 1] = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
        }
        return;
    }
    const bool second = d0 >= half;
    const int f = second ? d0 - half : d0, o = second ? d0 - half : d0 + half;
    const uint2 v = __ldg(reinterpret_cast<const uint2 *>(row + o));
    const float y[4] = {bf16_f32((uint16_t)v.x), bf16_f32((uint16_t)(v.x >> 16)), bf16_f32((uint16_t)v.y),
                        bf16_f32((uint16_t)(v.y >> 16))};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float c = __ldg(ct + f + i), s = __ldg(st + f + i);
        x[i] = second ? __fadd_rn(__fmul_rn(x[i], c), __fmul_rn(y[i], s)) : __fsub_rn(__fmul_rn(x[i], c), __fmul_rn(y[i], s));
    }
}

// ---------------------------------------------------------------------------
// the cached context
// ---------------------------------------------------------------------------

struct Shared {
    uint64_t full[kStages], empty[kStages];            // K and V tile loaded / both consumed
    uint64_t s_full[2], s_empty[2];                    // scores in tensor memory / read
    uint64_t p_full[2], pv_done[2];                    // weights in shared memory / their product added
    uint64_t q_full, v_full, drain;
    int64_t pre[kMaxReq + 1];                          // first tile of every request
    int64_t wsum[kThreads / 32];
    float2 scale[kScaleRing][kTile / 32];              // K and V scale of a tile's blocks
    float cf[kCols], mref[kCols], delta[kCols];        // score factor, reference maximum, its last raise (log2)
    float red[8][kCols];                               // per softmax warp
    uint32_t tmem;
    int32_t abort;
};

constexpr int kKBytes = kTile * kD;                    // one K or V tile: 16 KB
constexpr int kOffK = 0;
constexpr int kOffV = kOffK + kStages * kKBytes;
constexpr int kOffV16 = kOffV + kStages * kKBytes;     // [2 token halves][128 d][64 tokens] F16
constexpr int kOffP = kOffV16 + 2 * kKBytes;           // [2][kCols / 16 slabs][128 tokens][16] F16
constexpr int kPBytes = kCols * kTile * 2;
constexpr int kOffQ = kOffP + 2 * kPBytes;             // [3 pieces][kCols][128] E4M3
constexpr int kQBytes = kCols * kD;
constexpr int kOffShared = kOffQ + 3 * kQBytes;
constexpr int kSmem = kOffShared + (int)sizeof(Shared) + 1024;
static_assert(kPBytes % 1024 == 0 && kQBytes % 1024 == 0, "operand tiles keep their swizzle atoms aligned");
static_assert(kSmem <= 227 * 1024, "one CTA per SM");

constexpr uint32_t kTmS = 0, kTmO = 256, kTmCols = 512;   // scores at columns 0 and 128, sums at 256

// a stretch of tiles t0 .. t1 - 1 of one segment
struct Seg {
    int r, h, len, lo, rows, row0, nrows, t0, t1;
};

// the segment that tile `at` lies in, up to tile `end` of the whole list
__device__ __forceinline__ Seg segment(const AttnParams &p, const int64_t *pre, int64_t at, int64_t end)
{
    int a = 0, b = p.n_req;                 // pre[a] <= at < pre[b]
    while (b - a > 1) {
        const int m = (a + b) >> 1;
        if (pre[m] <= at) a = m;
        else b = m;
    }
    Seg s;
    s.r = a;
    s.lo = p.off[a];
    s.rows = p.off[a + 1] - s.lo;
    s.len = p.len[a];
    const int nt = (s.len + kTile - 1) / kTile;
    const int g = group_count(s.rows, p.G), per = group_rows(s.rows, p.G);
    const int64_t i = at - pre[a];
    const int seg = (int)(i / nt);
    s.t0 = (int)(i % nt);
    s.t1 = (int)min((int64_t)nt, s.t0 + (end - at));
    s.h = seg / g;
    s.row0 = seg % g * per;
    s.nrows = min(per, s.rows - s.row0);
    return s;
}

__device__ __forceinline__ bool bar_or(int id, int threads, bool x)
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %3, 0;\n\tbarrier.cta.red.or.pred q, %1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(r)
                 : "r"(id), "r"(threads), "r"((uint32_t)x)
                 : "memory");
    return r != 0;
}

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi)
{
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

// Reduce 16 columns over the 32 lanes of a warp: afterwards every lane holds
// the result of column lane_col(lane).  16 shuffles instead of 80.
__device__ __forceinline__ int lane_col(int lane)
{
    return ((lane & 1) << 3) | ((lane & 2) << 1) | ((lane & 4) >> 1) | ((lane & 8) >> 3);
}

template <bool kMax>
__device__ __forceinline__ float reduce16(const float *x, int lane)
{
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const bool up = lane & 1;
        const float o = __shfl_xor_sync(0xffffffffu, up ? x[i] : x[i + 8], 1), k = up ? x[i + 8] : x[i];
        v[i] = kMax ? fmaxf(k, o) : k + o;
    }
#pragma unroll
    for (int n = 4, bit = 2; n; n >>= 1, bit <<= 1) {
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const bool up = lane & bit;
            const float o = __shfl_xor_sync(0xffffffffu, up ? v[i] : v[i + n], bit), k = up ? v[i + n] : v[i];
            v[i] = kMax ? fmaxf(k, o) : k + o;
        }
    }
    const float o = __shfl_xor_sync(0xffffffffu, v[0], 16);
    return kMax ? fmaxf(v[0], o) : v[0] + o;
}

__global__ void __launch_bounds__(kThreads, 1)
    k_attn_ctx(const __grid_constant__ CUtensorMap kmap, const AttnParams p)
{
    extern __shared__ uint8_t raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~static_cast<uintptr_t>(1023));
    Shared &s = *reinterpret_cast<Shared *>(sm + kOffShared);
    const uint32_t base = smem_u32(sm);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int cta = blockIdx.x;
    auto bar = [&](const uint64_t &b) { return smem_u32(&b); };

    // ---- the tile list: tiles of every request, summed up
    int64_t mine = 0;
    if (tid < p.n_req) {
        int lo, rows, len;
        if (request_ok(p, tid, lo, rows, len))
            mine = rows ? (int64_t)((len + kTile - 1) / kTile) * p.H * group_count(rows, p.G) : 0;
        else
            fail(p.status);
    }
    int64_t incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t t = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += t;
    }
    if (lane == 31) s.wsum[warp] = incl;
    if (tid == 0) {
        s.abort = 0;
        for (int i = 0; i < kStages; ++i) {
            mbar_init(bar(s.full[i]), 1);
            mbar_init(bar(s.empty[i]), 2);               // scores computed, values widened
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(s.s_full[i]), 1);
            mbar_init(bar(s.s_empty[i]), kSoft / 32);
            mbar_init(bar(s.p_full[i]), kSoft / 32);
            mbar_init(bar(s.pv_done[i]), 1);
        }
        mbar_init(bar(s.q_full), kSoft / 32);
        mbar_init(bar(s.v_full), 1);
        mbar_init(bar(s.drain), 1);
        fence_mbar_init();
        prefetch_tmap(&kmap);
    }
    if (warp == 1) tmem_alloc(smem_u32(&s.tmem), kTmCols);
    __syncthreads();
    for (int w = 0; w < warp; ++w) incl += s.wsum[w];
    if (tid < p.n_req) s.pre[tid + 1] = incl;
    if (tid == 0) s.pre[0] = 0;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s.tmem;
    const int64_t total = s.pre[p.n_req];
    if (cta == 0 && tid <= p.n_req) p.plan[tid] = s.pre[tid];
    if (cta == 0 && tid == 0 && p.n_req == kThreads) p.plan[p.n_req] = total;
    const int64_t share = (total + p.ctas - 1) / p.ctas;
    const int64_t first = min(total, cta * share), end = min(total, first + share);
    const int nb = kTile / p.bt;                          // blocks of a tile
    volatile int32_t *abort = &s.abort;
    const uint64_t to = p.timeout_ns;

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        // Block numbers and scales are fetched 32 blocks at a time, one batch
        // ahead of their copies.
        uint32_t j = 0;
        bool ok = true;
        for (int64_t at = first; at < end && ok;) {
            const Seg g = segment(p, s.pre, at, end);
            const int b0 = g.t0 * nb, b1 = min((g.len + p.bt - 1) / p.bt, g.t1 * nb);
            const int32_t *table = p.table + (int64_t)g.r * p.max_blocks;
            int blk = 0;
            float2 sc = make_float2(0.f, 0.f);
            auto fetch = [&](int b, int &id, float2 &v) {
                id = 0;
                v = make_float2(0.f, 0.f);
                if (b < b1) {
                    id = __ldg(table + b);
                    if (id < 0 || id >= p.n_blocks) {
                        fail(p.status);
                        id = 0;
                    }
                    const int64_t i = (int64_t)id * p.H + g.h;
                    v = make_float2(__ldg(p.ks + i), __ldg(p.vs + i));
                }
            };
            fetch(b0 + lane, blk, sc);
            for (int b = b0; b < b1 && ok; b += 32) {
                int blk2;
                float2 sc2;
                fetch(b + 32 + lane, blk2, sc2);
                for (int l = 0; l < 32 && b + l < b1; l += nb, ++j) {
                    const int st = j % kStages;
                    ok = __all_sync(0xffffffffu, j < kStages || mbar_wait(bar(s.empty[st]), (j / kStages - 1) & 1, to,
                                                                          p.status, abort));
                    if (!ok) break;
                    const int n = min(nb, b1 - (b + l));      // blocks of this tile that hold tokens
                    const bool in = lane >= l && lane < l + nb;
                    if (in) s.scale[j % kScaleRing][lane - l] = sc;
                    __syncwarp();
                    if (lane == 0) mbar_expect_tx(bar(s.full[st]), (uint32_t)(n * p.bt * kD * 2));
                    __syncwarp();
                    if (in && lane < l + n) {
                        const int row = (blk * p.H + g.h) * p.bt;
                        tma_load_2d(base + kOffK + st * kKBytes + (lane - l) * p.bt * kD, &kmap, 0, row, bar(s.full[st]));
                        bulk_g2s(base + kOffV + st * kKBytes + (lane - l) * p.bt * kD, p.vc + (int64_t)row * kD,
                                 (uint32_t)(p.bt * kD), bar(s.full[st]));
                    }
                    __syncwarp();
                }
                blk = blk2;
                sc = sc2;
            }
            at += g.t1 - g.t0;
        }
        if (!ok) {                                            // copies in flight land before the CTA leaves
            const uint64_t t0 = globaltimer();
            for (uint32_t i = j > kStages ? j - kStages : 0; i < j; ++i)
                while (!mbar_try_wait_sleep(bar(s.full[i % kStages]), (i / kStages) & 1, kWaitSleepNs))
                    if (globaltimer() - t0 > to) break;
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA
        if (lane == 0) {
            uint32_t j = 0, q = 0;
            bool ok = true;
            auto pv = [&](uint32_t i, bool fresh, uint32_t idesc) -> bool {
                const int b = i & 1;
                if (!mbar_wait(bar(s.p_full[b]), (i >> 1) & 1, to, p.status, abort)) return false;
                if (!mbar_wait(bar(s.v_full), i & 1, to, p.status, abort)) return false;
                tc_fence_after();
                const uint64_t pd = smem_desc_mn_sw32(base + kOffP + b * kPBytes, kTile * 32);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const uint64_t vd = smem_desc_sw128(base + kOffV16 + (k >> 2) * kKBytes + (k & 3) * 32);
                    tc_mma_ss_f16(tmem + kTmO, vd, pd + (uint64_t)(k * (512 >> 4)), idesc, !(fresh && k == 0));
                }
                tc_commit(bar(s.pv_done[b]));
                return true;
            };
            for (int64_t at = first; at < end && ok; ++q) {
                const Seg g = segment(p, s.pre, at, end);
                const int n = (g.nrows * p.G + 15) & ~15;
                const uint32_t i_qk = idesc_e4m3_f32(kTile, n), i_pv = idesc_f16_f32_bmn(kD, n);
                ok = mbar_wait(bar(s.q_full), q & 1, to, p.status, abort);
                for (int t = g.t0; t < g.t1 && ok; ++t, ++j) {
                    const int st = j % kStages, b = j & 1;
                    ok = mbar_wait(bar(s.full[st]), (j / kStages) & 1, to, p.status, abort) &&
                         (j < 2 || mbar_wait(bar(s.s_empty[b]), ((j >> 1) - 1) & 1, to, p.status, abort));
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int c = 0; c < 3; ++c)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            tc_mma_ss_f8(tmem + kTmS + b * 128, smem_desc_sw128(base + kOffK + st * kKBytes + k * 32),
                                         smem_desc_sw128(base + kOffQ + c * kQBytes + k * 32), i_qk, c + k > 0);
                    tc_commit(bar(s.s_full[b]));
                    tc_commit(bar(s.empty[st]));
                    if (t > g.t0) ok = pv(j - 1, t - 1 == g.t0, i_pv);
                }
                if (ok) ok = pv(j - 1, g.t1 - 1 == g.t0, i_pv);
                at += g.t1 - g.t0;
            }
            if (!ok) {                                        // products in flight end before tensor memory is freed
                tc_commit(bar(s.drain));
                const uint64_t t0 = globaltimer();
                while (!mbar_try_wait_sleep(bar(s.drain), 0, kWaitSleepNs))
                    if (globaltimer() - t0 > to) break;
            }
        }
        __syncwarp();
    } else if (warp >= 12) {
        // ------------------------------------------------------------ V to F16
        const int t128 = tid - 384;
        uint32_t j = 0;
        bool ok = true;
        const int cs = p.bt == 32 ? 1 : p.bt == 64 ? 2 : 3;   // log2 of the 16-token chunks of a row of a block
        for (int64_t at = first; at < end && ok;) {
            const Seg g = segment(p, s.pre, at, end);
            for (int t = g.t0; t < g.t1; ++t, ++j) {
                const int st = j % kStages;
                ok = mbar_wait(bar(s.full[st]), (j / kStages) & 1, to, p.status, abort) &&
                     (j < 1 || mbar_wait(bar(s.pv_done[(j - 1) & 1]), ((j - 1) >> 1) & 1, to, p.status, abort));
                if (bar_or(3, 128, !ok)) {
                    ok = false;
                    break;
                }
                const int valid = min(kTile, g.len - t * kTile);
                const uint8_t *src = sm + kOffV + st * kKBytes;
#pragma unroll
                for (int it = 0; it < 8; ++it) {
                    const int i = it * 128 + t128;
                    const int row = i >> cs, d = row & (kD - 1);             // row: (block, d)
                    const int tok = (row >> 7) * p.bt + (i & ((1 << cs) - 1)) * 16;
                    uint4 w = make_uint4(0, 0, 0, 0);
                    if (tok < valid) w = *reinterpret_cast<const uint4 *>(src + i * 16);
                    uint32_t x[4] = {w.x, w.y, w.z, w.w};
                    if (tok + 16 > valid)                                     // what lies past the last token is not a value
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const int left = valid - tok - 4 * c;
                            x[c] &= left >= 4 ? 0xFFFFFFFFu : left <= 0 ? 0u : (1u << (8 * left)) - 1u;
                        }
                    uint32_t y[8];
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        y[2 * c] = e4m3x2_f16x2(x[c] & 0xFFFFu);
                        y[2 * c + 1] = e4m3x2_f16x2(x[c] >> 16);
                    }
                    uint8_t *dst = sm + kOffV16 + (tok >> 6) * kKBytes + d * 128;
                    const int c = (tok & 63) >> 3;
                    *reinterpret_cast<uint4 *>(dst + ((c ^ (d & 7)) << 4)) = make_uint4(y[0], y[1], y[2], y[3]);
                    *reinterpret_cast<uint4 *>(dst + (((c + 1) ^ (d & 7)) << 4)) = make_uint4(y[4], y[5], y[6], y[7]);
                }
                fence_async_shared();
                named_bar(3, 128);
                if (t128 == 0) {
                    mbar_arrive(bar(s.empty[st]));
                    mbar_arrive(bar(s.v_full));
                }
            }
            at += g.t1 - g.t0;
        }
    } else if (warp >= 4) {
        // ------------------------------------------------------------ softmax
        const int sw = warp - 4, wg = sw >> 2, quad = warp & 3;
        const int tok = quad * 32 + lane;                     // this thread's token of the tile
        const uint32_t lanes = (uint32_t)(quad * 32) << 16;
        uint32_t j = 0;
        bool ok = true;
        for (int64_t at = first; at < end && ok;) {
            const Seg g = segment(p, s.pre, at, end);
            const int ncol = g.nrows * p.G, npad = (ncol + 15) & ~15;
            // ---- Q: turned, scaled to E4M3's range by a power of two, in three pieces
            named_bar(4, kSoft);                              // the last segment's columns are done with
            for (int n = sw; n < npad; n += 8) {
                float x[4] = {0.f, 0.f, 0.f, 0.f};
                float f = 0.f;
                if (n < ncol) {
                    const int row = g.lo + g.row0 + n / p.G;
                    int pos = g.len + (int)p.depth[row];
                    if (p.rope.rot && pos >= p.rope.max_pos) {
                        fail(p.status);
                        pos = 0;
                    }
                    rotated4(p.q + row * p.q_stride + (int64_t)(g.h * p.G + n % p.G) * kD, lane * 4, pos, p.rope, x);
                    float top = fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
#pragma unroll
                    for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
                    const float qs = block_scale(top), qi = 1.f / qs;
                    f = qs * p.scale2;
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[i] *= qi;
                }
                const uint32_t dst = (uint32_t)(n * kD + (((lane >> 2) ^ (n & 7)) << 4) + (lane & 3) * 4);
#pragma unroll
                for (int c = 0; c < 3; ++c) {
                    uint32_t w = 0;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t code = to_e4m3(x[i]);
                        w |= code << (8 * i);
                        x[i] -= e4m3_f32((uint8_t)code);
                    }
                    *reinterpret_cast<uint32_t *>(sm + kOffQ + c * kQBytes + dst) = w;
                }
                if (lane == 0) {
                    s.cf[n] = f;
                    s.mref[n] = 0.f;
                }
            }
            fence_async_shared();
            named_bar(4, kSoft);
            if (lane == 0) mbar_arrive(bar(s.q_full));

            // ---- tiles; this warpgroup's 16-column chunks: c0 .. c0 + nch - 1
            const int all = npad >> 4, half = (all + 1) >> 1;
            const int c0 = wg ? half : 0, nch = wg ? all - half : half;
            float l[kChunks * 16];
#pragma unroll
            for (int i = 0; i < kChunks * 16; ++i) l[i] = 0.f;
            float sref = 0.f;
            for (int t = g.t0; t < g.t1; ++t, ++j) {
                const int b = j & 1;
                const bool fresh = t == g.t0;
                ok = mbar_wait(bar(s.s_full[b]), (j >> 1) & 1, to, p.status, abort);
                __syncwarp();
                tc_fence_after();
                float y[kChunks * 16];
                uint32_t *yr = reinterpret_cast<uint32_t *>(y);
#pragma unroll
                for (int c = 0; c < kChunks; ++c)
                    if (c < nch) tmem_ld_x16(tmem + lanes + kTmS + b * 128 + (c0 + c) * 16, yr + c * 16);
                tmem_ld_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(s.s_empty[b]));
                // the block scales of the tile
                const float2 *sc = s.scale[j % kScaleRing];
                const float2 my = sc[tok / p.bt];
                float top_v = 0.f;
                for (int i = 0; i < nb; ++i) top_v = fmaxf(top_v, sc[i].y);
                top_v = fmaxf(top_v, 1e-30f);
                const bool live = t * kTile + tok < g.len;
                bool raise = fresh || top_v > kScaleRaise * sref;
                float top = -INFINITY;
#pragma unroll
                for (int c = 0; c < kChunks; ++c)
                    if (c < nch) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const int n = (c0 + c) * 16 + i;
                            float v = fmaf(y[c * 16 + i], s.cf[n] * my.x, -s.mref[n]);
                            v = live ? v : -INFINITY;
                            y[c * 16 + i] = v;
                            top = fmaxf(top, v);
                        }
                    }
                raise |= top > kRaise;
                // this tile's P buffer is free once the product of two tiles ago is done
                if (ok && j >= 2) ok = mbar_wait(bar(s.pv_done[b]), ((j >> 1) - 1) & 1, to, p.status, abort);
                if (bar_or(5 + wg, 128, raise || !ok)) {
                    // ---- raise the references (first tile: set them)
                    if (ok && !fresh) ok = mbar_wait(bar(s.pv_done[b ^ 1]), ((j - 1) >> 1) & 1, to, p.status, abort);
#pragma unroll
                    for (int c = 0; c < kChunks; ++c)
                        if (c < nch) {
                            const float m = reduce16<true>(y + c * 16, lane);
                            if (lane < 16) s.red[sw][c * 16 + lane_col(lane)] = m;
                        }
                    if (bar_or(5 + wg, 128, !ok)) {
                        ok = false;
                        break;
                    }
                    if (tok < nch * 16) {
                        float m = fmaxf(fmaxf(s.red[wg * 4][tok], s.red[wg * 4 + 1][tok]),
                                        fmaxf(s.red[wg * 4 + 2][tok], s.red[wg * 4 + 3][tok]));
                        if (!fresh) m = fmaxf(m, 0.f);
                        if (!(m > -INFINITY)) m = 0.f;
                        s.delta[c0 * 16 + tok] = m;
                        s.mref[c0 * 16 + tok] += m;
                    }
                    named_bar(5 + wg, 128);
                    const float ref = fresh || top_v > kScaleRaise * sref ? top_v : sref;
                    const float fs = fresh ? 0.f : sref / ref;
                    sref = ref;
                    tc_fence_after();
#pragma unroll
                    for (int c = 0; c < kChunks; ++c)
                        if (c < nch) {
                            float o[16];
                            uint32_t *r = reinterpret_cast<uint32_t *>(o);
                            const uint32_t ta = tmem + lanes + kTmO + (c0 + c) * 16;
                            if (!fresh) {
                                tmem_ld_x16(ta, r);
                                tmem_ld_wait();
                            }
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                const float dl = s.delta[(c0 + c) * 16 + i];
                                const float f = ex2(-dl);
                                y[c * 16 + i] -= dl;
                                l[c * 16 + i] *= f;
                                o[i] *= f * fs;
                            }
                            if (!fresh) tmem_st_x16(ta, r);
                        }
                    tmem_st_wait();
                    tc_fence_before();
                }
                // ---- weights
                const float rt = kHead * (my.y / sref);
                uint8_t *prow = sm + kOffP + b * kPBytes + tok * 32;
                const int sw_bit = (tok >> 2) & 1;
#pragma unroll
                for (int c = 0; c < kChunks; ++c)
                    if (c < nch) {
                        uint32_t w[8];
#pragma unroll
                        for (int i = 0; i < 16; i += 2) {
                            const float e0 = ex2(y[c * 16 + i]), e1 = ex2(y[c * 16 + i + 1]);
                            l[c * 16 + i] += e0;
                            l[c * 16 + i + 1] += e1;
                            w[i >> 1] = pack_f16x2(live ? e0 * rt : 0.f, live ? e1 * rt : 0.f);
                        }
                        uint4 *dst = reinterpret_cast<uint4 *>(prow + (c0 + c) * (kTile * 32));
                        dst[sw_bit] = make_uint4(w[0], w[1], w[2], w[3]);
                        dst[sw_bit ^ 1] = make_uint4(w[4], w[5], w[6], w[7]);
                    }
                fence_async_shared();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(s.p_full[b]));
            }
            // ---- the segment's sums
            const uint32_t jl = j - 1;
            if (ok) ok = mbar_wait(bar(s.pv_done[jl & 1]), (jl >> 1) & 1, to, p.status, abort);
            if (bar_or(4, kSoft, !ok)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const int64_t col0 = (int64_t)g.lo * p.Hq + (int64_t)(g.h * g.rows + g.row0) * p.G + (int64_t)cta * kCols;
            const float back = sref / kHead;
#pragma unroll
            for (int c = 0; c < kChunks; ++c)
                if (c < nch) {
                    float o[16];
                    tmem_ld_x16(tmem + lanes + kTmO + (c0 + c) * 16, reinterpret_cast<uint32_t *>(o));
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int n = (c0 + c) * 16 + i;
                        if (n < ncol) p.part[(col0 + n) * kD + tok] = o[i] * back;
                    }
                    const float x = reduce16<false>(l + c * 16, lane);
                    if (lane < 16) s.red[sw][c * 16 + lane_col(lane)] = x;
                }
            tc_fence_before();
            named_bar(5 + wg, 128);
            if (tok < nch * 16 && c0 * 16 + tok < ncol)
                p.ml[col0 + c0 * 16 + tok] =
                    make_float2(s.mref[c0 * 16 + tok], (s.red[wg * 4][tok] + s.red[wg * 4 + 1][tok]) +
                                                           (s.red[wg * 4 + 2][tok] + s.red[wg * 4 + 3][tok]));
            at += g.t1 - g.t0;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, kTmCols);
}

// ---------------------------------------------------------------------------
// the root paths, and the merge
// ---------------------------------------------------------------------------

// One CTA per row and key/value head; a warp takes a query head of the group at
// a time, four dimensions to a lane.
__global__ void __launch_bounds__(128) k_attn_join(const AttnParams p)
{
    extern __shared__ __align__(16) float smf[];
    float *sv = smf;                                    // [kPath][kD], read four at a time
    float *sq = sv + kPath * kD;                        // [4 warps][kD]
    float *sk = sq + 4 * kD;                            // [kPath][kD + 1] keys of the path, turned
    float *ss = sk + kPath * (kD + 1);                  // [4 warps][kPath] weights
    __shared__ int32_t s_parent[kMaxBudget], s_path[kPath + 1], s_n;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
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
            if (q >= j || (p.rope.rot && p.len[r] + (int)p.depth[j] >= p.rope.max_pos)) n = kPath + 1;   // a parent after its child, a position off the table
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
    const int len = p.len[r], rows = p.off[r + 1] - lo;
    for (int a = warp; a < nA; a += 4) {
        const int64_t j = s_path[a];
        float x[4];
        rotated4(p.k + j * p.k_stride + h * kD, lane * 4, len + (int)p.depth[j], p.rope, x);
#pragma unroll
        for (int i = 0; i < 4; ++i) sk[a * (kD + 1) + lane * 4 + i] = x[i];
        const uint2 w = __ldg(reinterpret_cast<const uint2 *>(p.v + j * p.v_stride + h * kD + lane * 4));
        *reinterpret_cast<float4 *>(sv + a * kD + lane * 4) =
            make_float4(bf16_f32((uint16_t)w.x), bf16_f32((uint16_t)(w.x >> 16)), bf16_f32((uint16_t)w.y),
                        bf16_f32((uint16_t)(w.y >> 16)));
    }
    __syncthreads();
    // the shares that hold a part of this row's segment
    pdl_wait();
    const int64_t total = __ldcg(p.plan + p.n_req), share = (total + p.ctas - 1) / p.ctas;
    const int nt = (len + kTile - 1) / kTile;
    const int i0 = row - lo, grp = i0 / group_rows(rows, G);
    const int64_t a0 = __ldcg(p.plan + r) + (int64_t)(h * group_count(rows, G) + grp) * nt;
    const int cta0 = nt ? (int)(a0 / share) : 0, cta1 = nt ? (int)((a0 + nt - 1) / share) : -1;
    for (int g = warp; g < G; g += 4) {
        float x[4];
        rotated4(p.q + row * p.q_stride + (int64_t)(h * G + g) * kD, lane * 4, len + (int)p.depth[row], p.rope, x);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i) sq[warp * kD + lane * 4 + i] = x[i] * p.scale2;
        __syncwarp();
        float m = -INFINITY;
        for (int a = lane; a < nA; a += 32) {
            float d0 = 0.f, d1 = 0.f;
#pragma unroll 8
            for (int d = 0; d < kD; d += 2) {
                d0 = fmaf(sq[warp * kD + d], sk[a * (kD + 1) + d], d0);
                d1 = fmaf(sq[warp * kD + d + 1], sk[a * (kD + 1) + d + 1], d1);
            }
            ss[warp * kPath + a] = d0 + d1;
            m = fmaxf(m, d0 + d1);
        }
        const int64_t col = (int64_t)lo * p.Hq + (int64_t)(h * rows + i0) * G + g;
        for (int c = cta0 + lane; c <= cta1; c += 32) m = fmaxf(m, __ldcg(p.ml + col + (int64_t)c * kCols).x);
#pragma unroll
        for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
        if (!(m > -INFINITY)) m = 0.f;                  // nothing but NaN and -inf: the sums say so
        __syncwarp();
        float l = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
        for (int a = 0; a < nA; ++a) {
            const float e = ex2(ss[warp * kPath + a] - m);
            const float4 v = *reinterpret_cast<const float4 *>(sv + a * kD + lane * 4);
            l += e;
            acc[0] = fmaf(e, v.x, acc[0]);
            acc[1] = fmaf(e, v.y, acc[1]);
            acc[2] = fmaf(e, v.z, acc[2]);
            acc[3] = fmaf(e, v.w, acc[3]);
        }
#pragma unroll 4
        for (int c = cta0; c <= cta1; ++c) {
            const float2 q = __ldcg(p.ml + col + (int64_t)c * kCols);
            const float4 v = __ldcg(reinterpret_cast<const float4 *>(p.part + (col + (int64_t)c * kCols) * kD) + lane);
            const float e = ex2(q.x - m);
            l = fmaf(e, q.y, l);
            acc[0] = fmaf(e, v.x, acc[0]);
            acc[1] = fmaf(e, v.y, acc[1]);
            acc[2] = fmaf(e, v.z, acc[2]);
            acc[3] = fmaf(e, v.w, acc[3]);
        }
        *reinterpret_cast<uint2 *>(o + g * kD + lane * 4) =
            make_uint2(pack_bf16x2(acc[0] / l, acc[1] / l), pack_bf16x2(acc[2] / l, acc[3] / l));
        __syncwarp();
    }
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn()
{
    static EncodeTiledFn fn = nullptr;
    if (!fn) {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(f);
    }
    return fn;
}

size_t plan_bytes() { return (size_t)((kMaxReq + 1) * 8 + 255) / 256 * 256; }
size_t part_columns(int32_t R, int32_t Hq, int ctas) { return (size_t)R * Hq + (size_t)ctas * kCols; }

}  // namespace

namespace w12i {

size_t attn_ws_bytes(int32_t R, int32_t Hq, int32_t H, int32_t n_req, int num_sms)
{
    (void)H;
    (void)n_req;
    return plan_bytes() + part_columns(R, Hq, num_sms) * (kD * 4 + 8);
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
    p.ctas = a.num_sms;
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
    uint8_t *w = static_cast<uint8_t *>(a.work);
    const size_t cols = part_columns(a.R, a.Hq, p.ctas);
    p.plan = reinterpret_cast<int64_t *>(w);
    p.part = reinterpret_cast<float *>(w + plan_bytes());
    p.ml = reinterpret_cast<float2 *>(w + plan_bytes() + cols * kD * 4);
    p.status = a.status;
    p.timeout_ns = a.timeout_ns;
    cudaStream_t st = static_cast<cudaStream_t>(stream);

    EncodeTiledFn fn = encode_fn();
    if (!fn) return (int)cudaErrorNotSupported;
    CUtensorMap kmap;
    const cuuint64_t dims[2] = {(cuuint64_t)kD, (cuuint64_t)a.n_blocks * a.H * a.bt};
    const cuuint64_t strides[1] = {(cuuint64_t)kD};
    const cuuint32_t box[2] = {(cuuint32_t)kD, (cuuint32_t)a.bt}, es[2] = {1, 1};
    if (fn(&kmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t *>(a.kc), dims, strides, box, es,
           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return (int)cudaErrorInvalidValue;
    cudaError_t e = cudaFuncSetAttribute(k_attn_ctx, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return (int)e;
    k_attn_ctx<<<p.ctas, kThreads, kSmem, st>>>(kmap, p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return (int)e;
    constexpr int smem = (kPath * (2 * kD + 1) + 4 * (kD + kPath)) * 4;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)a.R, (unsigned)a.H);
    cfg.blockDim = dim3(128);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return (int)cudaLaunchKernelEx(&cfg, k_attn_join, p);
}

}  // namespace w12i
