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
// request and many short ones balance alike.  Starting and ending a segment
// costs as much as a handful of tiles, so every segment has a lead of as many
// empty ones in the list, and a tile counts by its columns (kLead and
// tile_weight; 256 rows of 32 requests: the slowest CTA was 23% over the mean
// without the leads, 10% without the weights).  A share leaves, for every
// segment (request, head, group) that it meets, FP32 sums with their maximum
// and normaliser; k_attn_join merges them with the root path's.
//
// Tokens lie on the 128 lanes of tensor memory, query rows (rows x heads of
// the group, padded to 16) on its columns: few queries cost few columns, not
// an empty 128-row tile, and the cached codes are the A operand of both
// products, which is read once per tile whatever the number of queries.
//   S^T = K Q^T  kind::f8f6f4: K's codes as they lie in the cache; Q in three
//                E4M3 pieces that add up to twelve significant bits (2^-17 of
//                the head's largest at least).  Up to kStack columns the
//                pieces are stacked as further columns (a product costs the
//                tensor cores its A operand, so one of 48 columns is a third
//                of three of 16) and added up by the reader; above, each piece
//                is a product of its own into the same accumulators.
//   O^T = V^T P  kind::f16: V's codes widened to F16 (exact) by warpgroups of
//                their own, into tensor memory (through shared memory they
//                would cost four times the bandwidth, which bounds the tile);
//                P in F16, eleven significant bits down to 2^-16 of the
//                largest weight there was when its reference was set, and
//                multiples of 2^-26 of it below.
// Two groups of two softmax warpgroups take alternate tiles, each with its own
// scores, P, maxima and sums, so that the latencies of one tile's chain
// (product, reads, exponentials, vote, product) hide behind the other's; the
// warpgroups of a group share the tile's columns.  The groups merge at the end
// of a segment.  Scores come to the threads in the 16x256b fragments: a thread
// holds two columns of each eight and four tokens, so a column's factors, its
// maximum and its normaliser are registers (with a token to a thread they were
// four 16-byte loads of shared memory to eight columns, and those bound the
// pass), and P is stored by stmatrix.
// The maximum is lazy: P refers to a column maximum that is only raised when a
// score passes it by 2^6 (P stays under F16's top), so the usual tile has no
// reduction over lanes at all; the same slow path raises the reference of the
// value scales, which P carries.  A raise costs several tiles, so a reference
// is set 2^6 above the maximum: with normally distributed scores that leaves
// next to none but the first.  What P can hold below the reference is F16's
// range less those 2^12 and 2 for the value scales: every binade of margin less
// keeps weights half as large, but 32 rows behind 32771 tokens take 67 us with
// 2^5, 74 with 2^4 and 97 with 2^2 where they take 60 to 62 with 2^6.  Scores
// that rise along the context cost their raises: 152 rows of 64 heads behind
// 40000 tokens take 363 us flat, 369 rising by 2^30 in all and 478 by 2^300; of
// one head 224, 225 and 240; falling, nothing.
// A token that outweighs the others by 2^20 and more would leave them few bits
// or none, and if its own value is small they are the output.  So every 128
// tiles of a group a column whose scores have all come to lie far below its
// reference gets one of their own again: sums and normalisers are FP32 and can
// be scaled up.  At most 128 tiles' weights are then rounded to multiples of
// 2^-26 of a larger one: together 2^-13 of its weight at most.
//
// What bounds it.  One row behind a long context: memory (131072 tokens of 8
// heads, 268 MB: 55.6 us, 4.8 TB/s, of which the tiles' loop 46 us at 5.8).
// Many rows: the tensor cores' turn of a tile.  At M = 128 a product costs them
// some 75 to 130 cycles however few its columns, so a tile takes 1280 cycles at
// 16 columns, 1740 at 48 and 2250 at 80 (32 rows behind 32771 tokens: 60 to
// 62 us; 256 rows of 32 requests behind up to 16384: 198 us, 3.8 TB/s), and a
// segment's start and end some 8000 to 23000 more.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>

#include "w12_device.cuh"
#include "w12_kv.cuh"

namespace {

using namespace w12d;
using namespace w12i;

constexpr int kD = kKvDim;
constexpr int kPath = kMaxDepth + 1;       // rows of a root path
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kTile = 128;                 // tokens of a tile
constexpr int kStack = 48;                 // columns up to which Q's pieces are stacked
constexpr int kMaxCols = 80;               // query columns of a segment, see Shape
constexpr int kScaleRing = 16;             // tiles whose block scales are kept (the copies run at most 8 ahead of their readers)
constexpr int kMaxReq = kMaxBudget;
constexpr int kLead = 9;                   // a segment's start and end in tiles: 7 of 16 columns, 10 of 48 and 80
constexpr uint64_t kDrainNs = 1000000000;  // limit of the waits after a failed one
constexpr int kSoft = 512;                 // softmax threads, in four warpgroups
constexpr int kThreads = 128 + kSoft + 256; // warps: 0 K copies, 1 scores, 2 V copies, 3 sums, 4-19 softmax, 20-27 V to F16
// Registers a thread: at launch, of the softmax warps, of the others.  The
// shares add up to no more than the launch has (a larger one would wait for
// ever).  Shared memory leaves the L1 cache so little that a spilled register
// is a read of L2: the shapes of 16 and 48 columns spill none, that of 80 five
// (20 bytes stored, 28 read).
constexpr int kRegsLaunch = 72, kRegsSoft = 88, kRegsOther = 48;
static_assert(kSoft * kRegsSoft + (kThreads - kSoft) * kRegsOther <= kThreads * kRegsLaunch, "register shares");
constexpr float kHead = 256.f;             // P of a weight of 1 under the reference scale
constexpr float kMargin = 6.f;             // a reference is set this (log2) above the largest score there was
constexpr float kRaise = 6.f;              // a score may pass the column's reference by this (log2) before it is raised
constexpr float kCap = 8.f;                // scores are held under this until then
constexpr float kScaleRaise = 2.f;         // ... and a value scale its reference by this factor: 256 * 2^6 * 2 = 2^15 < F16's top
// Every kSettle tiles of a group the references of columns whose scores have
// all fallen kFar below come down again, to kLower under their highest at most.
constexpr int kSettle = 128;
constexpr float kFar = -12.f, kLower = 40.f;

struct AttnParams {
    int32_t H, Hq, G, bt, n_blocks, max_blocks, n_req, R, ctas;
    int32_t cols, fit;                      // query columns of a segment at most; rows of so many
    int64_t q_stride, k_stride, v_stride;
    const uint8_t *kc, *vc;
    const float *ks, *vs;
    const int32_t *table, *len, *off, *parent, *req;
    const uint8_t *depth;
    const uint16_t *q, *k, *v;
    RopeArgs rope;
    float scale2;                           // softmax scale * log2(e)
    uint16_t *out;
    float *part;                            // [R * Hq + ctas * cols][kD] sums
    float2 *ml;                             // [R * Hq + ctas * cols] maximum (log2), normaliser
    int32_t *status;
    uint64_t timeout_ns;                    // a wait's limit
    int32_t debug_flags;                    // bit 0: CTA 0 never copies a key (test hook)
};

__device__ __forceinline__ void fail(int32_t *status) { atomicCAS(status, 0, (int32_t)W12_E_INVAL); }

// rows of a request's groups: as many as fit the columns, evenly
__device__ __forceinline__ int group_count(int rows, int fit) { return (rows + fit - 1) / fit; }
// what a tile of such a request counts in the split: 0.35 us and 0.13 us for every 16 columns
__device__ __forceinline__ int tile_weight(const AttnParams &p, int rows)
{
    const int g = group_count(rows, p.fit);
    return 11 + 4 * (((rows + g - 1) / g * p.G + 15) >> 4);
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

// What requests have in the list: tiles, the same weighted, weighted segments.
struct List {
    int64_t tiles, units;
    int32_t segs;
    __device__ __forceinline__ void add(const List &o) { tiles += o.tiles, units += o.units, segs += o.segs; }
};

__device__ __forceinline__ List list_of(const AttnParams &p, int rows, int len)
{
    List l{0, 0, 0};
    if (rows > 0 && len > 0) {
        const int w = tile_weight(p, rows), segs = p.H * group_count(rows, p.fit);
        l.tiles = (int64_t)((len + kTile - 1) / kTile) * segs;
        l.units = l.tiles * w;
        l.segs = segs * w;
    }
    return l;
}

// How the whole list is cut: the lead of a segment, and whether tiles are
// weighted.  Every CTA starts one segment, whatever it does.  A lead counts
// where it goes on to another, and would only waste shares of a few tiles;
// those are also too small for weights (a share has to have a tile of every
// segment that it lies in).
struct Cut {
    int32_t lead;
    bool weighted;
    __device__ __forceinline__ Cut(const AttnParams &p, const List &all)
    {
        lead = (int32_t)min((uint32_t)kLead, (uint32_t)min(all.tiles, (int64_t)INT32_MAX) / (4u * p.ctas));   // (no 64-bit division)
        weighted = lead > 0 && all.units + (int64_t)lead * all.segs <= INT32_MAX;
        if (!weighted) lead = 0;
    }
    __device__ __forceinline__ int64_t length(const List &l) const { return weighted ? l.units + (int64_t)lead * l.segs : l.tiles; }
};

// Four consecutive elements d0 .. d0 + 3 of a BF16 row and what turns them by
// position pos; loaded apart from the arithmetic, so that the loads of several
// rows are in flight together.  The rotated part is a multiple of 8 wide, so a
// pair's two halves lie in two such groups, or in one with adjacent pairs.
struct Raw4 {
    uint2 w, v;                             // the elements, their partners
    float4 c, s;
};

__device__ __forceinline__ void load4(Raw4 &x, const uint16_t *row, int d0, int pos, const RopeArgs &r)
{
    x.w = __ldg(reinterpret_cast<const uint2 *>(row + d0));
    x.v = make_uint2(0, 0);
    x.c = make_float4(1.f, 1.f, 1.f, 1.f);
    x.s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (d0 >= r.rot) return;
    const int half = r.rot >> 1;
    const int64_t t = (int64_t)pos * half;
    if (r.adjacent) {
        x.v = make_uint2((x.w.x >> 16) | (x.w.x << 16), (x.w.y >> 16) | (x.w.y << 16));
        const float2 c = __ldg(reinterpret_cast<const float2 *>(r.cos + t + (d0 >> 1)));
        const float2 s = __ldg(reinterpret_cast<const float2 *>(r.sin + t + (d0 >> 1)));
        x.c = make_float4(c.x, c.x, c.y, c.y);
        x.s = make_float4(-s.x, s.x, -s.y, s.y);
    } else {
        const bool second = d0 >= half;
        const int o = second ? d0 - half : d0 + half, f = second ? o : d0;
        x.v = __ldg(reinterpret_cast<const uint2 *>(row + o));
        x.c = __ldg(reinterpret_cast<const float4 *>(r.cos + t + f));
        x.s = __ldg(reinterpret_cast<const float4 *>(r.sin + t + f));
        if (!second) x.s = make_float4(-x.s.x, -x.s.y, -x.s.z, -x.s.w);
    }
}

__device__ __forceinline__ float4 turn4(const Raw4 &r)
{
    return make_float4(__fadd_rn(__fmul_rn(bf16_lo(r.w.x), r.c.x), __fmul_rn(bf16_lo(r.v.x), r.s.x)),
                       __fadd_rn(__fmul_rn(bf16_hi(r.w.x), r.c.y), __fmul_rn(bf16_hi(r.v.x), r.s.y)),
                       __fadd_rn(__fmul_rn(bf16_lo(r.w.y), r.c.z), __fmul_rn(bf16_lo(r.v.y), r.s.z)),
                       __fadd_rn(__fmul_rn(bf16_hi(r.w.y), r.c.w), __fmul_rn(bf16_hi(r.v.y), r.s.w)));
}

// Wait for a phase: false after about timeout_ns (W12_E_TIMEOUT in *status) or
// once *abort is set.  try_wait without a time hint parks the warp in hardware;
// with one it becomes a loop of sleeps, and twenty warps' sleep loops took more
// issue slots here than the work did.  The clock and the abort word are looked
// at every 256th time.
__device__ __forceinline__ bool wait_phase(uint32_t bar, uint32_t parity, uint64_t timeout_ns, int32_t *status,
                                           volatile int32_t *abort)
{
    uint64_t t0 = 0;
    for (uint32_t n = 1; !mbar_try_wait(bar, parity); ++n) {
        if (n & 255) continue;
        const uint64_t t = globaltimer();
        if (t0 == 0) t0 = t;
        const bool late = t - t0 > timeout_ns;
        if (late) atomicCAS(status, 0, (int32_t)W12_E_TIMEOUT);
        if (late || *abort) {
            *abort = 1;
            return false;
        }
    }
    return true;
}

// ---------------------------------------------------------------------------
// the cached context
// ---------------------------------------------------------------------------

// What a launch is compiled for: the query columns of a segment.  A request
// with more gets several groups of rows, each reading the context again (from
// L2, side by side), so any shape serves any tree; the host picks the least
// one that holds an average request's.  Fewer columns leave shared memory for
// more tiles in flight.
template <int kCols>
struct Shape {
    static constexpr int kChunks = kCols / 16;
    static constexpr bool kStacked = kCols <= kStack;
    static constexpr int kSteps = kChunks;                       // steps of 8 columns of a softmax warpgroup, at most
    static constexpr int kStK = kCols <= 16 ? 6 : 5;             // K tiles in flight
    static constexpr int kStV = kCols <= 16 ? 6 : kCols <= 48 ? 5 : 4;
    static constexpr int kKBytes = kTile * kD;                   // one K or V tile: 16 KB
    static constexpr int kPBytes = kCols * kTile * 2;
    static constexpr int kQBytes = kCols * kD;
    static constexpr int kOffK = 0;
    static constexpr int kOffV = kOffK + kStK * kKBytes;
    static constexpr int kOffP = kOffV + kStV * kKBytes;         // [2][kCols / 16 slabs][128 tokens][16] F16
    static constexpr int kOffQ = kOffP + 2 * kPBytes;            // [3 pieces][kCols][128] E4M3
    static constexpr int kOffShared = kOffQ + 3 * kQBytes;
    // tensor memory: scores of two tiles, sums of the two groups, two V tiles in F16 (two tokens to a column)
    static constexpr int kTmS = kStacked ? 3 * kCols : kCols;    // columns of one tile's scores
    static constexpr int kTmO = 2 * kTmS;
    static constexpr int kTmV = kTmO + 2 * kCols;
    static constexpr int kTmUsed = kTmV + kTile;
    static constexpr int kTmCols = kTmUsed <= 256 ? 256 : 512;
    static_assert(kTmUsed <= 512, "tensor memory");
};

constexpr int kMaxStages = 6;
constexpr int kRowBits = 10;                                 // of a request's row count

struct Shared {
    uint64_t k_full[kMaxStages], k_empty[kMaxStages];  // K and V tiles loaded / consumed
    uint64_t v_full[kMaxStages], v_empty[kMaxStages];
    uint64_t s_full[2], s_empty[2];                    // scores in tensor memory / read
    uint64_t p_full[2], v16_full[2], pv_done[2];       // weights and widened values in shared memory / their product added
    uint64_t q_full, drain[2];
    int32_t pre[kMaxReq + 1];                          // where every request starts in the list
    int32_t lead, weighted;
    alignas(16) float cf[kMaxCols];                    // score factor of a column
    alignas(16) float mneg[2][kMaxCols];               // per group: minus its reference maximum,
    alignas(16) float delta[2][kMaxCols];              // the factor of its last raise; at the end, of the group's sums
    union {
        alignas(16) float red[2][4][kMaxCols];         // per warp
        List list[kThreads / 32];                      // before: a warp's requests
    };
    union {
        float mtop[2][kMaxCols];                       // the highest reference that a column ever had
        float lsum[2][kMaxCols];                       // at the end: normalisers
    };
    float sref[2];
    int32_t len[kMaxReq];                              // of every request: cached tokens,
    uint16_t lo[kMaxReq], rows[kMaxReq];               // first row; rows, and above kRowBits the weight of its tiles
    float2 scale[kScaleRing][kTile / 32];              // K and V scale of a tile's blocks
    float top_v[kScaleRing];                           // the largest of the V scales
    uint32_t tmem;
    int32_t abort;
};

template <int kCols>
constexpr int smem_bytes()
{
    return Shape<kCols>::kOffShared + (int)sizeof(Shared) + 1024;
}
static_assert(smem_bytes<16>() <= 227 * 1024 && smem_bytes<48>() <= 227 * 1024 && smem_bytes<80>() <= 227 * 1024,
              "one CTA per SM");


// a stretch of tiles t0 .. t1 - 1 of one segment
struct Seg {
    int r, h, len, lo, rows, row0, nrows, t0, t1;
};

// the next segment with tiles in at .. end - 1 of the list, up to `end`; `at` moves behind it
__device__ __forceinline__ bool next_segment(const AttnParams &p, const Shared &sh, int32_t &at, int32_t end, Seg &s)
{
    while (at < end) {
        int a = 0;                          // pre[a] <= at < pre[a + 1]
        for (int step = 512; step; step >>= 1)
            if (a + step < p.n_req && sh.pre[a + step] <= at) a += step;
        s.r = a;
        s.lo = sh.lo[a];
        s.rows = sh.rows[a];
        s.len = sh.len[a];
        const uint32_t w = sh.weighted ? s.rows >> kRowBits : 1;
        s.rows &= (1 << kRowBits) - 1;
        const uint32_t n = ((uint32_t)(s.len + kTile - 1) / kTile + sh.lead) * w;
        const int g = group_count(s.rows, p.fit), per = (s.rows + g - 1) / g;
        const uint32_t i = (uint32_t)(at - sh.pre[a]), seg = i / n, u0 = i - seg * n;
        const uint32_t u1 = min(n, u0 + (uint32_t)(end - at));
        at += (int32_t)(u1 - u0);
        s.t0 = max((int)((u0 + w - 1) / w) - sh.lead, 0);     // a tile is its first unit's
        s.t1 = (int)((u1 + w - 1) / w) - sh.lead;
        s.h = (int)(seg / (uint32_t)g);
        s.row0 = (int)(seg % (uint32_t)g) * per;
        s.nrows = min(per, s.rows - s.row0);
        if (s.t0 < s.t1) return true;
    }
    return false;
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

// the machine's 2^x, within 2^-22 of it; results under 2^-126 are zero
__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// two FP32 operations at a time
__device__ __forceinline__ uint64_t pair(float a, float b)
{
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ void unpair(uint64_t d, float &a, float &b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(d)); }
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

// the larger, or NaN
__device__ __forceinline__ float max_nan(float a, float b)
{
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

// 32 lanes x 8 columns as two fragments of 16 lanes: thread t gets columns
// 2 (t % 4) and the next of lanes t / 4 + 8 i in y[2 i], y[2 i + 1]
__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, float *y)
{
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x1.b32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(y[0]), "=f"(y[1]), "=f"(y[2]), "=f"(y[3])
                 : "r"(taddr));
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x1.b32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(y[4]), "=f"(y[5]), "=f"(y[6]), "=f"(y[7])
                 : "r"(taddr + (16u << 16)));
}

// four 8x8 matrices of 16-bit values, rows at the lanes' addresses
__device__ __forceinline__ void stsm_x4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d)
                 : "memory");
}

// 32 lanes x 8 columns
__device__ __forceinline__ void tmem_ld_x8(uint32_t taddr, float *r)
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7])
                 : "r"(taddr));
}

// the loads before it are complete, and these registers of theirs are read after it only
__device__ __forceinline__ void ld_done8(float *y)
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(y[0]), "+f"(y[1]), "+f"(y[2]), "+f"(y[3]), "+f"(y[4]), "+f"(y[5]), "+f"(y[6]), "+f"(y[7]));
}

__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(
            taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

__device__ __forceinline__ void tmem_st_x8(uint32_t taddr, const float *r)
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "f"(r[0]),
                 "f"(r[1]), "f"(r[2]), "f"(r[3]), "f"(r[4]), "f"(r[5]), "f"(r[6]), "f"(r[7])
                 : "memory");
}

template <int N>
__device__ __forceinline__ void regs_inc()
{
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_dec()
{
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi)
{
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

template <int kCols>
__global__ void __launch_bounds__(kThreads, 1)
    k_attn_ctx(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap, const AttnParams p)
{
    typedef Shape<kCols> T;
    extern __shared__ uint8_t raw[];
    uint8_t *sm = raw + (-smem_u32(raw) & 1023u);         // (arithmetic that leaves the compiler sure of shared memory)
    Shared &s = *reinterpret_cast<Shared *>(sm + T::kOffShared);
    const uint32_t base = smem_u32(sm);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int cta = blockIdx.x;
    auto bar = [&](const uint64_t &b) { return smem_u32(&b); };

    pdl_launch_dependents();                              // the join may start wherever there is room
    // ---- the tile list: tiles of every request, summed up
    List incl{0, 0, 0};
    if (tid < p.n_req) {
        int lo, rows, len;
        if (!request_ok(p, tid, lo, rows, len)) {
            rows = 0;
            fail(p.status);
        }
        incl = list_of(p, rows, len);
        s.lo[tid] = (uint16_t)lo;
        s.rows[tid] = (uint16_t)(rows | (rows ? tile_weight(p, rows) : 1) << kRowBits);
        s.len[tid] = len;
    }
    auto scan = [&](List &l) {                            // over a warp
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const List o{__shfl_up_sync(0xffffffffu, l.tiles, d), __shfl_up_sync(0xffffffffu, l.units, d), __shfl_up_sync(0xffffffffu, l.segs, d)};
            if (lane >= d) l.add(o);
        }
    };
    auto from = [&](const List &l, int i) -> List {
        return {__shfl_sync(0xffffffffu, l.tiles, i), __shfl_sync(0xffffffffu, l.units, i), __shfl_sync(0xffffffffu, l.segs, i)};
    };
    if (warp * 32 < p.n_req) scan(incl);
    if (tid == 96) {                                      // (a warp that has nothing else to do here)
        s.abort = 0;
        for (int i = 0; i < kMaxStages; ++i) {
            mbar_init(bar(s.k_full[i]), 1);
            mbar_init(bar(s.k_empty[i]), 1);
            mbar_init(bar(s.v_full[i]), 1);
            mbar_init(bar(s.v_empty[i]), 4);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(s.s_full[i]), 1);
            mbar_init(bar(s.s_empty[i]), kSoft / 64);
            mbar_init(bar(s.p_full[i]), kSoft / 64);
            mbar_init(bar(s.v16_full[i]), 4);
            mbar_init(bar(s.pv_done[i]), 1);
        }
        mbar_init(bar(s.q_full), kSoft / 32);
        mbar_init(bar(s.drain[0]), 1);
        mbar_init(bar(s.drain[1]), 1);
        fence_mbar_init();
        prefetch_tmap(&kmap);
        prefetch_tmap(&vmap);
    }
    if (warp == 1) tmem_alloc(smem_u32(&s.tmem), T::kTmCols);
    List all;
    const bool one = p.n_req <= 32;                       // one warp has all requests
    if (one) {
        all = from(incl, 31);
    } else {                                              // what the warps before had, and all
        static_assert(kThreads / 32 <= 32, "a warp's sums to a lane");
        if (lane == 31) s.list[warp] = incl;
        __syncthreads();
        all = lane * 32 < p.n_req ? s.list[lane] : List{0, 0, 0};
        scan(all);
        if (warp) incl.add(from(all, warp - 1));
        all = from(all, 31);
    }
    if (!one || warp == 0) {
        const Cut cut(p, all);
        const bool fits = cut.length(all) <= INT32_MAX;   // else there is nothing to do but say so
        if (!fits && tid == 0) atomicCAS(p.status, 0, (int32_t)W12_E_UNSUPPORTED);
        if (tid < p.n_req) s.pre[tid + 1] = fits ? (int32_t)cut.length(incl) : 0;
        if (tid == 0) s.pre[0] = 0, s.lead = cut.lead, s.weighted = cut.weighted;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s.tmem;
    const int32_t total = s.pre[p.n_req];
    const int64_t share = ((uint32_t)total + p.ctas - 1) / p.ctas;
    const int32_t first = (int32_t)min((int64_t)total, cta * share), end = (int32_t)min((int64_t)total, first + share);
    const int bs = p.bt == 32 ? 5 : p.bt == 64 ? 6 : 7;   // log2 of a block's tokens
    const int nb = kTile >> bs;                           // blocks of a tile
    volatile int32_t *abort = &s.abort;
    const uint64_t to = p.timeout_ns;
    // after a wait that ran out: products in flight end before tensor memory is freed
    auto drain = [&](const uint64_t &b) {
        tc_commit(bar(b));
        const uint64_t t0 = globaltimer();
        while (!mbar_try_wait_sleep(bar(b), 0, kWaitSleepNs))
            if (globaltimer() - t0 > kDrainNs) break;
    };

    if (warp == 0 || warp == 2) {
        // ------------------------------------------------------------ copies: warp 0 K and the block scales, warp 2 V
        // Block numbers (and scales) are fetched 32 blocks at a time, one
        // batch ahead of their copies.  A thread's loop of wait, expect and
        // copy takes some 200 ns a turn, so K and V have one each.
        regs_dec<kRegsOther>();
        const bool is_k = warp == 0;
        const int stages = is_k ? T::kStK : T::kStV;
        const uint32_t full = smem_u32(is_k ? s.k_full : s.v_full), empty = smem_u32(is_k ? s.k_empty : s.v_empty);
        const uint32_t tile0 = base + (is_k ? T::kOffK : T::kOffV), bytes = (uint32_t)(p.bt * kD);
        uint32_t j = 0, st = 0, par = 1;                      // tile, its stage, the parity its stage's last use left
        bool ok = true;
        Seg g;
        const bool withheld = is_k && cta == 0 && (p.debug_flags & 1);
        for (int32_t at = withheld ? end : first; ok && next_segment(p, s, at, end, g);) {
            const int b0 = g.t0 * nb, b1 = min((g.len + p.bt - 1) >> bs, g.t1 * nb);
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
                    if (is_k) v = make_float2(__ldg(p.ks + i), __ldg(p.vs + i));
                }
            };
            fetch(b0 + lane, blk, sc);
            for (int b = b0; b < b1 && ok; b += 32) {
                int blk2;
                float2 sc2;
                fetch(b + 32 + lane, blk2, sc2);
                const int row = is_k ? (blk * p.H + g.h) << bs : (blk * p.H + g.h) * kD;   // of the pool seen as rows
                for (int l = 0; l < 32 && b + l < b1; l += nb, ++j) {
                    const int n = min(nb, b1 - (b + l));      // blocks of this tile that hold tokens
                    const bool in = lane >= l && lane < l + nb;
                    const uint32_t f = full + st * 8;
                    ok = __all_sync(0xffffffffu, wait_phase(empty + st * 8, par, to, p.status, abort));
                    if (!ok) break;
                    // the copies first: a segment's first scales are still on their
                    // way, and the phase stays open until this warp's arrival
                    if (in && lane < l + n) {
                        const uint32_t dst = tile0 + st * T::kKBytes + (uint32_t)(lane - l) * bytes;
                        tma_load_2d(dst, is_k ? &kmap : &vmap, 0, row, f);
                    }
                    if (is_k) {
                        float top = sc.y;                     // the tile's largest V scale
                        for (int d = 1; d < nb; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
                        if (in) s.scale[j % kScaleRing][lane - l] = sc;
                        if (lane == l) s.top_v[j % kScaleRing] = top;
                    }
                    __syncwarp();
                    if (lane == l) mbar_expect_tx(f, n * bytes);
                    if (++st == (uint32_t)stages) st = 0, par ^= 1;
                }
                blk = blk2;
                sc = sc2;
            }
        }
        if (!ok) {                                            // copies in flight land before the CTA leaves
            const uint64_t t0 = globaltimer();
            for (uint32_t i = j >= (uint32_t)stages ? j - stages : 0; i < j; ++i)
                while (!mbar_try_wait_sleep(full + i % stages * 8, (i / stages) & 1, kWaitSleepNs))
                    if (globaltimer() - t0 > kDrainNs) break;
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ scores: S^T = K Q^T
        regs_dec<kRegsOther>();
        if (lane == 0) {
            uint32_t j = 0, q = 0, st = 0, par = 0;
            bool ok = true;
            const uint64_t kd = smem_desc_sw128(base + T::kOffK), qd = smem_desc_sw128(base + T::kOffQ);
            Seg g;
            for (int32_t at = first; ok && next_segment(p, s, at, end, g); ++q) {
                const int n = (g.nrows * p.G + 15) & ~15;
                const uint32_t idesc = idesc_e4m3_f32(kTile, T::kStacked ? 3 * kCols : n);
                ok = wait_phase(bar(s.q_full), q & 1, to, p.status, abort);
                for (int t = g.t0; t < g.t1 && ok; ++t, ++j) {
                    const int b = j & 1;
                    ok = (j < 2 || wait_phase(bar(s.s_empty[b]), ((j >> 1) - 1) & 1, to, p.status, abort)) &&
                         wait_phase(bar(s.k_full[st]), par, to, p.status, abort);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t ka = kd + (uint64_t)(st * (T::kKBytes >> 4));
#pragma unroll
                    for (int c = 0; c < (T::kStacked ? 1 : 3); ++c)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            tc_mma_ss_f8(tmem + b * T::kTmS, ka + k * 2, qd + (uint64_t)((c * T::kQBytes + k * 32) >> 4), idesc, c + k > 0);
                    tc_commit(bar(s.s_full[b]));
                    tc_commit(bar(s.k_empty[st]));
                    if (++st == T::kStK) st = 0, par ^= 1;
                }
            }
            if (!ok) drain(s.drain[0]);
        }
        __syncwarp();
    } else if (warp == 3) {
        // ------------------------------------------------------------ sums: O^T += V^T P
        regs_dec<kRegsOther>();
        if (lane == 0) {
            uint32_t j = 0;
            bool ok = true;
            const uint64_t pd = smem_desc_mn_sw32(base + T::kOffP, kTile * 32);
            Seg g;
            for (int32_t at = first; ok && next_segment(p, s, at, end, g);) {
                const uint32_t idesc = idesc_f16_f32_bmn(kD, (g.nrows * p.G + 15) & ~15);
                for (int t = g.t0; t < g.t1 && ok; ++t, ++j) {
                    const int b = j & 1;
                    ok = wait_phase(bar(s.v16_full[b]), (j >> 1) & 1, to, p.status, abort) &&
                         wait_phase(bar(s.p_full[b]), (j >> 1) & 1, to, p.status, abort);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t keep = t - g.t0 >= 2;      // each group's first tile starts its sums
                    const uint64_t pb = pd + (uint64_t)(b * (T::kPBytes >> 4));
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        tc_mma_ts(tmem + T::kTmO + b * kCols, tmem + T::kTmV + b * (kTile / 2) + k * 8, pb + (uint64_t)(k * (512 >> 4)),
                                  idesc, keep | (k > 0));
                    tc_commit(bar(s.pv_done[b]));
                }
            }
            if (!ok) drain(s.drain[1]);
        }
        __syncwarp();
    } else if (warp >= 20) {
        // ------------------------------------------------------------ V to F16
        regs_dec<kRegsOther>();
        const int wg = (warp - 20) >> 2, quad = warp & 3, d = quad * 32 + lane;   // a dimension to a thread, as the lanes lie
        const int cs = bs - 4;                                // log2 of the 16-token chunks of a row of a block
        const int swz = bs == 5 ? (d >> 2) & 1 : bs == 6 ? (d >> 1) & 3 : d & 7;   // the copy's swizzle: one row's bytes wide
        const uint32_t dst = tmem + ((uint32_t)(quad * 32) << 16) + T::kTmV + wg * (kTile / 2);
        uint32_t j = 0;
        bool ok = true;
        Seg g;
        for (int32_t at = first; ok && next_segment(p, s, at, end, g);) {
            for (int t = g.t0; t < g.t1; ++t, ++j) {
                if ((int)(j & 1) != wg) continue;
                const int st = j % T::kStV;
                ok = __all_sync(0xffffffffu, wait_phase(bar(s.v_full[st]), (j / T::kStV) & 1, to, p.status, abort) &&
                                                 (j < 2 || wait_phase(bar(s.pv_done[wg]), ((j >> 1) - 1) & 1, to, p.status, abort)));
                if (!ok) break;
                tc_fence_after();
                const int valid = min(kTile, g.len - t * kTile);
                const uint8_t *src = sm + T::kOffV + st * T::kKBytes + (d << bs);
#pragma unroll 1
                for (int part = 0; part < 4; ++part) {
                    uint32_t y[16];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int c = part * 2 + i;                           // chunk c of the tile's eight
                        const int blk = c >> cs, in = c & ((1 << cs) - 1);
                        const uint4 w = *reinterpret_cast<const uint4 *>(src + ((blk * kD) << bs) + ((in ^ swz) << 4));
                        y[i * 8] = e4m3x2_f16x2(w.x & 0xFFFFu), y[i * 8 + 1] = e4m3x2_f16x2(w.x >> 16);
                        y[i * 8 + 2] = e4m3x2_f16x2(w.y & 0xFFFFu), y[i * 8 + 3] = e4m3x2_f16x2(w.y >> 16);
                        y[i * 8 + 4] = e4m3x2_f16x2(w.z & 0xFFFFu), y[i * 8 + 5] = e4m3x2_f16x2(w.z >> 16);
                        y[i * 8 + 6] = e4m3x2_f16x2(w.w & 0xFFFFu), y[i * 8 + 7] = e4m3x2_f16x2(w.w >> 16);
                    }
                    if (part * 32 + 32 > valid) {                             // what lies past the last token is not a value
                        const int left = valid - part * 32;
#pragma unroll
                        for (int i = 0; i < 16; ++i) y[i] = 2 * i + 1 < left ? y[i] : 2 * i < left ? y[i] & 0xFFFFu : 0u;
                    }
                    tmem_st_x16(dst + part * 16, y);
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(bar(s.v_empty[st]));
                    mbar_arrive(bar(s.v16_full[wg]));
                }
            }
        }
    } else if (warp >= 4) {
        // ------------------------------------------------------------ softmax: group grp takes the tiles j with j % 2 == grp,
        // its two warpgroups half of the columns each
        regs_inc<kRegsSoft>();
        const int sw = warp - 4, wg = sw >> 2, quad = warp & 3, grp = wg >> 1;
        const int tok = quad * 32 + lane;                     // this thread's token of the tile
        const uint32_t tm = tmem + ((uint32_t)(quad * 32) << 16);
        uint32_t j = 0;
        bool ok = true;
        Seg g;
        for (int32_t at = first; ok && next_segment(p, s, at, end, g);) {
            const int ncol = g.nrows * p.G, npad = (ncol + 15) & ~15;
            const int col0 = g.lo * p.Hq + (g.h * g.rows + g.row0) * p.G + cta * kCols;   // its columns in the workspace
            // ---- Q: turned, scaled to E4M3's range by a power of two, in three pieces
            named_bar(4, kSoft);                              // the last segment's columns are done with
            const int n_q = T::kStacked ? kCols : npad;       // stacked pieces are products of all their columns
            // A column ahead, its depth two: their loads are in flight while a column is split.
            constexpr int kStep = kSoft / 32;
            Raw4 rw;
            auto place = [&](int n, int &row, int &head) {
                const int i = min(n, ncol - 1);
                row = g.lo + g.row0 + i / p.G;
                head = g.h * p.G + i % p.G;
            };
            auto fetch = [&](int row, int head, int depth) {
                int pos = g.len + depth;
                if (p.rope.rot && pos >= p.rope.max_pos) {
                    fail(p.status);
                    pos = 0;
                }
                load4(rw, p.q + (int64_t)row * p.q_stride + (int64_t)head * kD, lane * 4, pos, p.rope);
            };
            int row, head, row2, head2;
            place(sw, row, head);
            place(sw + kStep, row2, head2);
            int depth = __ldg(p.depth + row), depth2 = __ldg(p.depth + row2);
            if (sw < n_q) fetch(row, head, depth);
#pragma unroll 1
            for (int n = sw; n < n_q; n += kStep) {
                float4 x = turn4(rw);
                if (n + kStep < n_q) {
                    fetch(row2, head2, depth2);
                    place(n + 2 * kStep, row2, head2);
                    depth2 = __ldg(p.depth + row2);
                }
                float top = fmaxf(fmaxf(fabsf(x.x), fabsf(x.y)), fmaxf(fabsf(x.z), fabsf(x.w)));
#pragma unroll
                for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
                const float qs = block_scale(top), f = n < ncol ? 1.f / qs : 0.f;
                // infinities have no code: the column becomes NaN, as their products would
                const float qi = top < INFINITY ? f : __int_as_float(0x7FC00000);
                x = make_float4(x.x * qi, x.y * qi, x.z * qi, x.w * qi);
                const uint32_t dst = (uint32_t)(n * kD + (((lane >> 2) ^ (n & 7)) << 4) + (lane & 3) * 4);
#pragma unroll
                for (int c = 0; c < 3; ++c) {
                    const uint32_t lo = to_e4m3x2(x.x, x.y), hi = to_e4m3x2(x.z, x.w);
                    *reinterpret_cast<uint32_t *>(sm + T::kOffQ + c * T::kQBytes + dst) = lo | (hi << 16);
                    const float2 a = f16x2_f32(e4m3x2_f16x2(lo)), b = f16x2_f32(e4m3x2_f16x2(hi));
                    x = make_float4(x.x - a.x, x.y - a.y, x.z - b.x, x.w - b.y);
                }
                if (lane == 0) {
                    s.cf[n] = n < ncol ? qs * p.scale2 : 0.f;
                    s.mneg[0][n] = 0.f;
                    s.mneg[1][n] = 0.f;
                    s.mtop[0][n] = s.mtop[1][n] = -INFINITY;
                }
            }
            fence_async_shared();
            named_bar(4, kSoft);
            if (lane == 0) mbar_arrive(bar(s.q_full));

            // ---- this warpgroup's columns, 8 to a step, two of them this thread's
            const int all = npad >> 3, steps = all >> 1, s0 = (wg & 1) * steps, n0 = s0 * 8, my_n = n0 + (lane & 3) * 2;
            uint64_t cf[T::kSteps], mneg[T::kSteps], l[T::kSteps];
#pragma unroll
            for (int c = 0; c < T::kSteps; ++c)
                if (c < steps) {
                    cf[c] = *reinterpret_cast<const uint64_t *>(s.cf + my_n + c * 8);
                    mneg[c] = l[c] = 0ull;
                }
            float sref = 0.f, inv_ref = 0.f;
            bool fresh = true;
            const uint32_t j0 = j;
            j += g.t1 - g.t0;
            const int left0 = g.len - g.t0 * kTile - quad * 32 - (lane >> 2);   // tokens from this thread's first on
            const uint32_t tm_s = tm + grp * T::kTmS + n0, tm_o = tm + T::kTmO + grp * kCols + n0;
            const uint32_t prow = base + T::kOffP + grp * T::kPBytes + tok * 32, flip = (tok >> 2) & 1;
            for (uint32_t jj = j0 + ((j0 ^ grp) & 1); jj < j; jj += 2) {
                ok = wait_phase(bar(s.s_full[grp]), (jj >> 1) & 1, to, p.status, abort);
                // the group's P and sums are free once its last product is done
                if (ok && jj >= 2) ok = wait_phase(bar(s.pv_done[grp]), ((jj >> 1) - 1) & 1, to, p.status, abort);
                __syncwarp();
                tc_fence_after();
                const float2 my = s.scale[jj % kScaleRing][(quad * 32) >> bs];   // of the block that this warp's 32 tokens lie in
                const float top_v = fmaxf(s.top_v[jj % kScaleRing], 1e-30f);
                const int valid = left0 - (int)(jj - j0) * kTile;                // token i of this thread's four is there if 8 i < valid
                const uint64_t ks2 = pair(my.x, my.x);
                // a step's scores against the references, in log2 units
                auto scores = [&](int c, float *y) {
                    tmem_ld_frag(tm_s + c * 8, y);
                    float y1[T::kStacked ? 8 : 1], y2[T::kStacked ? 8 : 1];
                    if constexpr (T::kStacked) {
                        tmem_ld_frag(tm_s + kCols + c * 8, y1);
                        tmem_ld_frag(tm_s + 2 * kCols + c * 8, y2);
                        ld_done8(y1);
                        ld_done8(y2);
                    }
                    ld_done8(y);
                    const uint64_t f = mul2(cf[c], ks2);
#pragma unroll
                    for (int i = 0; i < 8; i += 2) {
                        uint64_t a = pair(y[i], y[i + 1]);
                        if constexpr (T::kStacked) a = add2(a, add2(pair(y1[i], y1[i + 1]), pair(y2[i], y2[i + 1])));
                        unpair(fma2(a, f, mneg[c]), y[i], y[i + 1]);
                    }
                };
                // The tile's weights into P and the normalisers; returns the
                // largest score, over kRaise if the references have to be
                // raised first.  Until then scores are held under kCap, which
                // also stands for a NaN; a dead token's under everything.
                auto weights = [&](float sign) -> float {
                    const float rt = my.y * inv_ref;
                    const uint64_t rt2 = pair(rt, rt), sg2 = pair(sign, sign);
                    float cap[4], top = -INFINITY;
#pragma unroll
                    for (int i = 0; i < 4; ++i) cap[i] = 8 * i < valid ? kCap : -INFINITY;
#pragma unroll
                    for (int c = 0; c < T::kSteps; ++c)
                        if (c < steps) {
                            float y[8];
                            scores(c, y);
                            uint32_t w[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const float x0 = fminf(y[2 * i], cap[i]), x1 = fminf(y[2 * i + 1], cap[i]);
                                top = fmaxf(fmaxf(top, x0), x1);
                                const uint64_t e = pair(ex2(x0), ex2(x1));
                                l[c] = fma2(e, sg2, l[c]);
                                float u, v;
                                unpair(mul2(e, rt2), u, v);
                                w[i] = pack_f16x2(u, v);
                            }
                            const uint32_t sc = s0 + c;
                            stsm_x4(prow + (sc >> 1) * (kTile * 32) + (((sc & 1) ^ flip) << 4), w[0], w[1], w[2], w[3]);
                        }
                    return top;
                };
                // Raise the references (first tile: set them).  A column with a
                // NaN among its scores gets a NaN for its raise, and so carries
                // it into its normaliser and sums.
                auto raise = [&](bool must, bool settle) -> bool {
#pragma unroll
                    for (int c = 0; c < T::kSteps; ++c)
                        if (c < steps) {
                            float y[8];
                            scores(c, y);
                            float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                if (8 * i < valid) m0 = max_nan(m0, y[2 * i]), m1 = max_nan(m1, y[2 * i + 1]);
#pragma unroll
                            for (int d = 4; d < 32; d <<= 1) {
                                m0 = max_nan(m0, __shfl_xor_sync(0xffffffffu, m0, d));
                                m1 = max_nan(m1, __shfl_xor_sync(0xffffffffu, m1, d));
                            }
                            if (lane < 4) *reinterpret_cast<float2 *>(&s.red[grp][quad][my_n + c * 8]) = make_float2(m0, m1);
                        }
                    if (bar_or(5 + wg, 128, !ok)) return false;
                    if (tok < steps * 8) {
                        const int n = n0 + tok;
                        float m = max_nan(max_nan(s.red[grp][0][n], s.red[grp][1][n]), max_nan(s.red[grp][2][n], s.red[grp][3][n]));
                        float ref = -s.mneg[grp][n];
                        if (m == -INFINITY || (!fresh && m <= kRaise && !(settle && m < kFar))) {
                            m = 0.f;
                        } else {
                            m = max_nan(m + kMargin, s.mtop[grp][n] - kLower - ref);
                            ref += m;
                            s.mneg[grp][n] = -ref;
                            s.mtop[grp][n] = fmaxf(s.mtop[grp][n], ref);
                        }
                        s.delta[grp][n] = fresh ? 1.f : ex2(-m);   // (nothing to scale yet, and 2^-m may be no number)
                    }
                    named_bar(5 + wg, 128);
                    const float ref = must ? top_v : sref, fs = sref / ref;
                    sref = ref;
                    inv_ref = kHead / ref;
#pragma unroll
                    for (int c = 0; c < T::kSteps; ++c)
                        if (c < steps) {
                            l[c] = mul2(l[c], *reinterpret_cast<const uint64_t *>(&s.delta[grp][my_n + c * 8]));
                            mneg[c] = *reinterpret_cast<const uint64_t *>(&s.mneg[grp][my_n + c * 8]);
                        }
                    if (!fresh) {
#pragma unroll 1
                        for (int c = 0; c < steps; ++c) {
                            float o[8];
                            tmem_ld_x8(tm_o + c * 8, o);
                            ld_done8(o);
#pragma unroll
                            for (int i = 0; i < 8; ++i) o[i] *= s.delta[grp][n0 + c * 8 + i] * fs;
                            tmem_st_x8(tm_o + c * 8, o);
                        }
                        tmem_st_wait();
                    }
                    return true;
                };
                // Once over the scores, as a rule; where a score passes its
                // reference, once more to take the weights back, and again
                // under raised references.  One copy of the pass serves all three.
                const bool must = fresh || top_v > kScaleRaise * sref;          // the same for every thread
                const bool settle = (jj - j0) % (2 * kSettle) >= 2 * kSettle - 2;
                for (int turn = must || settle ? 2 : 0;; ++turn) {
                    if (turn == 2 && !raise(must, settle)) {
                        ok = false;
                        break;
                    }
                    const float top = weights(turn == 1 ? -1.f : 1.f);
                    if (turn == 2 || (turn == 0 && !bar_or(5 + wg, 128, top > kRaise || !ok))) break;
                }
                if (!ok) break;
                fresh = false;
                tc_fence_before();
                fence_async_shared();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(bar(s.s_empty[grp]));
                    mbar_arrive(bar(s.p_full[grp]));
                }
            }
            // ---- the segment's sums: each group's normalisers, then both groups' sums merged
            const uint32_t last = j - 1 - ((j - 1 - grp) & 1);     // the last tile of this group's parity, if it had one
            if (ok && !fresh) ok = wait_phase(bar(s.pv_done[grp]), (last >> 1) & 1, to, p.status, abort);
            if (bar_or(4, kSoft, !ok)) {
                ok = false;
                break;
            }
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < T::kSteps; ++c)
                if (c < steps) {
                    float x, y;
                    unpair(l[c], x, y);
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) {
                        x += __shfl_xor_sync(0xffffffffu, x, d);
                        y += __shfl_xor_sync(0xffffffffu, y, d);
                    }
                    if (lane < 4) *reinterpret_cast<float2 *>(&s.red[grp][quad][my_n + c * 8]) = make_float2(x, y);
                }
            named_bar(5 + wg, 128);
            if (tok < steps * 8) {
                const int n = n0 + tok;
                s.lsum[grp][n] = (s.red[grp][0][n] + s.red[grp][1][n]) + (s.red[grp][2][n] + s.red[grp][3][n]);
                if (fresh) s.mneg[grp][n] = INFINITY;          // no maximum: the group had no tile
            }
            if (tok == 0) s.sref[grp] = sref;
            named_bar(4, kSoft);
            // a group without a tile has left no sums: whatever stands there counts for nothing
            const bool has0 = s.sref[0] > 0.f, has1 = s.sref[1] > 0.f;
            if (wg == 0 && tok < npad) {
                const float m0 = -s.mneg[0][tok], m1 = -s.mneg[1][tok], m = max_nan(m0, m1);
                const float f0 = has0 ? ex2(m0 - m) : 0.f, f1 = has1 ? ex2(m1 - m) : 0.f;
                s.delta[0][tok] = f0 * s.sref[0] / kHead;
                s.delta[1][tok] = f1 * s.sref[1] / kHead;
                if (tok < ncol) p.ml[col0 + tok] = make_float2(m, (has0 ? f0 * s.lsum[0][tok] : 0.f) + (has1 ? f1 * s.lsum[1][tok] : 0.f));
            }
            named_bar(4, kSoft);
#pragma unroll 1
            for (int c = wg; c < all; c += 4) {
                float o0[8], o1[8];
                tmem_ld_x8(tm + T::kTmO + c * 8, o0);
                tmem_ld_x8(tm + T::kTmO + kCols + c * 8, o1);
                ld_done8(o0);
                ld_done8(o1);
                float *dst = p.part + (int64_t)(col0 + c * 8) * kD + tok;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (c * 8 + i < ncol)
                        dst[i * kD] = (has0 ? o0[i] * s.delta[0][c * 8 + i] : 0.f) + (has1 ? o1[i] * s.delta[1][c * 8 + i] : 0.f);
            }
            tc_fence_before();
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, T::kTmCols);
}

// ---------------------------------------------------------------------------
// the root paths, and the merge
// ---------------------------------------------------------------------------

// One CTA per row and key/value head; a warp takes a query head of the group at
// a time, four dimensions to a lane.  It starts with the context's kernel (where
// an SM has room) and waits for it after the path's scores.  Bound by the
// latency of its loads: so many small CTAs to an SM, everything asked for as
// soon as its address is known (parents and depths of all rows up to this one
// before its request is), and a context's parts fetched four at a time with
// their maxima.
constexpr int kJoinWarps = 8;                           // at most; as many as the group has heads
constexpr int kJoinKey = kD + 4;                        // stride of a key
constexpr int kJoinParts = 4;

__global__ void __launch_bounds__(kJoinWarps * 32, 4) k_attn_join(const AttnParams p)
{
    __shared__ __align__(16) float sk[kPath * kJoinKey];      // keys of the path, turned
    __shared__ __align__(16) uint2 sv[kPath][kD / 4];         // its values, as they come
    __shared__ __align__(16) float sq[kJoinWarps][kD];
    __shared__ float ss[kJoinWarps][kPath + 3];               // scores
    __shared__ int32_t s_parent[kMaxBudget], s_path[kPath + 1], s_n;
    __shared__ uint8_t s_depth[kMaxBudget];
    __shared__ int32_t s_cta0, s_cta1;                        // the shares that hold a part of this row's segment
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, threads = blockDim.x, warps = threads >> 5;
    const int row = blockIdx.x, h = blockIdx.y, G = p.G;
    int r = p.req[row];
    for (int j = tid; j <= row; j += threads) {
        s_parent[j] = p.parent[j];
        s_depth[j] = p.depth[j];
    }
    int lo = 0, rows = 1, len = 0;
    if (r < 0 || r >= p.n_req || !request_ok(p, r, lo, rows, len) || row < lo || row >= lo + rows)
        r = -1, lo = row, rows = 1, len = 0;
    __syncthreads();
    // a position on the table (or none)
    auto placed = [&](int j) { return p.rope.rot == 0 || len + (int)s_depth[j] < p.rope.max_pos; };
    const bool served = r >= 0 && placed(row);
    Raw4 rw;
    if (served && warp < G)
        load4(rw, p.q + row * p.q_stride + (int64_t)(h * G + warp) * kD, lane * 4, len + (int)s_depth[row], p.rope);
    if (warp == 0) {
        int n = 0, j = row;
        while (served && j >= lo && n <= kPath) {
            if (lane == 0) s_path[n] = j;
            ++n;
            const int q = s_parent[j];
            if (q >= j) n = kPath + 1;                  // a parent after its child
            else j = q;
        }
        const bool ok = served && n <= kPath && j < 0;  // ... or outside the request
        bool off = false;                               // a position off the table
        __syncwarp();
        if (ok)
            for (int a = lane; a < n; a += 32) off |= !placed(s_path[a]);
        off = __any_sync(0xffffffffu, off);
        if (lane == 0) {
            s_n = ok && !off ? n : 0;
            if (!ok || off) fail(p.status);
        }
    }
    const int ng = group_count(rows, p.fit), per = (rows + ng - 1) / ng, i0 = row - lo, grp = i0 / per;
    if (warp == warps - 1) {                            // the list again, as k_attn_ctx cuts it
        List all{0, 0, 0}, before{0, 0, 0};
        for (int i = lane; i < p.n_req; i += 32) {
            int l, n, c;
            if (!request_ok(p, i, l, n, c)) continue;
            const List mine = list_of(p, n, c);
            all.add(mine);
            if (i < r) before.add(mine);
        }
        auto sum = [&](List &l) {
#pragma unroll
            for (int d = 16; d; d >>= 1)
                l.add({__shfl_xor_sync(0xffffffffu, l.tiles, d), __shfl_xor_sync(0xffffffffu, l.units, d), __shfl_xor_sync(0xffffffffu, l.segs, d)});
        };
        sum(all);
        sum(before);
        const Cut cut(p, all);
        const int64_t total = cut.length(all), share = max((int64_t)1, (total + p.ctas - 1) / p.ctas);
        const int nt = total <= INT32_MAX ? (len + kTile - 1) / kTile : 0, w = cut.weighted ? tile_weight(p, rows) : 1;
        const int64_t a0 = cut.length(before) + ((int64_t)(h * ng + grp) * (nt + cut.lead) + cut.lead) * w;
        if (lane == 0) {
            s_cta0 = (int)(a0 / share);
            s_cta1 = nt ? (int)((a0 + (int64_t)(nt - 1) * w) / share) : -1;
        }
    }
    __syncthreads();
    const int nA = s_n;
    uint16_t *o = p.out + ((int64_t)row * p.Hq + h * G) * kD;
    if (nA == 0) {                                      // malformed: zeros, and the status word says so
        for (int i = tid; i < G * kD; i += threads) o[i] = 0;
        pdl_wait();                                     // a call is over when its context's kernel is, whatever its rows
        return;
    }
    for (int a = warp; a < nA; a += warps) {
        const int64_t j = s_path[a];
        Raw4 kw;
        load4(kw, p.k + j * p.k_stride + h * kD, lane * 4, len + (int)s_depth[j], p.rope);
        sv[a][lane] = __ldg(reinterpret_cast<const uint2 *>(p.v + j * p.v_stride + h * kD + lane * 4));
        *reinterpret_cast<float4 *>(sk + a * kJoinKey + lane * 4) = turn4(kw);
    }
    __syncthreads();
    bool waited = false;
    for (int g = warp; g < G; g += warps) {
        if (g >= warps)                                 // (the first is on its way)
            load4(rw, p.q + row * p.q_stride + (int64_t)(h * G + g) * kD, lane * 4, len + (int)s_depth[row], p.rope);
        const float4 x = turn4(rw);
        __syncwarp();
        *reinterpret_cast<float4 *>(&sq[warp][lane * 4]) =
            make_float4(x.x * p.scale2, x.y * p.scale2, x.z * p.scale2, x.w * p.scale2);
        __syncwarp();
        // scores: eight lanes to a row of the path, sixteen dimensions each
        float4 q[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) q[i] = *reinterpret_cast<const float4 *>(&sq[warp][(lane & 7) * 4 + i * 32]);
        float m = -INFINITY;
        for (int a = lane >> 3; a < kPath + 3; a += 4) {
            if (a - (lane >> 3) >= nA) break;
            float y = 0.f;
            if (a < nA) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float4 k = *reinterpret_cast<const float4 *>(sk + a * kJoinKey + (lane & 7) * 4 + i * 32);
                    y = fmaf(q[i].x, k.x, fmaf(q[i].y, k.y, fmaf(q[i].z, k.z, fmaf(q[i].w, k.w, y))));
                }
            }
#pragma unroll
            for (int d = 4; d; d >>= 1) y += __shfl_xor_sync(0xffffffffu, y, d);
            if (a < nA) {
                if ((lane & 7) == 0) ss[warp][a] = y;
                m = fmaxf(m, y);
            }
        }
#pragma unroll
        for (int d = 16; d >= 8; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
        m = fmaxf(m, -1e30f);                           // (nothing but NaN and -inf: the sums say so)
        __syncwarp();
        float l = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
        auto add = [&](float e, float n, const float4 &v) {
            l = fmaf(e, n, l);
            acc[0] = fmaf(e, v.x, acc[0]);
            acc[1] = fmaf(e, v.y, acc[1]);
            acc[2] = fmaf(e, v.z, acc[2]);
            acc[3] = fmaf(e, v.w, acc[3]);
        };
        for (int a = 0; a < nA; ++a) {
            const uint2 v = sv[a][lane];
            add(ex2(ss[warp][a] - m), 1.f, make_float4(bf16_lo(v.x), bf16_hi(v.x), bf16_lo(v.y), bf16_hi(v.y)));
        }
        if (!waited) pdl_wait();                        // the context's parts from here on
        waited = true;
        const int cta0 = s_cta0, cta1 = s_cta1;
        const int64_t col = (int64_t)lo * p.Hq + (int64_t)(h * rows + i0) * G + g;
        for (int c = cta0; c <= cta1; c += kJoinParts) {
            float2 ml[kJoinParts];
            float4 v[kJoinParts];
#pragma unroll
            for (int i = 0; i < kJoinParts; ++i)
                if (c + i <= cta1) {
                    const int64_t at = col + (int64_t)(c + i) * p.cols;
                    ml[i] = __ldcg(p.ml + at);
                    v[i] = __ldcg(reinterpret_cast<const float4 *>(p.part + at * kD) + lane);
                }
            const float old = m;
#pragma unroll
            for (int i = 0; i < kJoinParts; ++i)
                if (c + i <= cta1) m = fmaxf(m, ml[i].x);
            const float f = ex2(old - m);
            l *= f;
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[i] *= f;
#pragma unroll
            for (int i = 0; i < kJoinParts; ++i)
                if (c + i <= cta1) add(ex2(ml[i].x - m), ml[i].y, v[i]);
        }
        const float i = 1.f / l;
        *reinterpret_cast<uint2 *>(o + g * kD + lane * 4) =
            make_uint2(pack_bf16x2(acc[0] * i, acc[1] * i), pack_bf16x2(acc[2] * i, acc[3] * i));
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

// Registers a thread of a shape's kernel, looked up once per shape; 0 if that
// failed (and then looked up again).
template <int kCols>
int ctx_registers()
{
    static std::atomic<int> known{0};
    int n = known.load(std::memory_order_relaxed);
    if (n == 0) {
        cudaFuncAttributes f{};
        if (cudaFuncGetAttributes(&f, k_attn_ctx<kCols>) == cudaSuccess) known.store(n = f.numRegs, std::memory_order_relaxed);
    }
    return n;
}

template <int kCols>
cudaError_t launch_ctx(const CUtensorMap &kmap, const CUtensorMap &vmap, const AttnParams &p, cudaStream_t st)
{
    constexpr int bytes = smem_bytes<kCols>();
    const cudaError_t e = cudaFuncSetAttribute(k_attn_ctx<kCols>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    if (ctx_registers<kCols>() < kRegsLaunch) return cudaErrorInvalidConfiguration;   // the register shares need that many
    k_attn_ctx<kCols><<<p.ctas, kThreads, bytes, st>>>(kmap, vmap, p);
    return cudaGetLastError();
}

size_t part_columns(int32_t R, int32_t Hq, int ctas) { return (size_t)R * Hq + (size_t)ctas * kMaxCols; }

}  // namespace

namespace w12i {

size_t attn_ws_bytes(int32_t R, int32_t Hq, int32_t H, int32_t n_req, int num_sms)
{
    (void)H;
    (void)n_req;
    return part_columns(R, Hq, num_sms) * (kD * 4 + 8);
}

int attn_registers(int cols, int *wanted)
{
    *wanted = kRegsLaunch;
    return cols == 16 ? ctx_registers<16>() : cols == 48 ? ctx_registers<48>() : cols == 80 ? ctx_registers<80>() : 0;
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
    p.part = reinterpret_cast<float *>(w);
    p.ml = reinterpret_cast<float2 *>(w + cols * kD * 4);
    p.status = a.status;
    p.timeout_ns = a.timeout_ns;
    p.debug_flags = a.debug_flags;
    cudaStream_t st = static_cast<cudaStream_t>(stream);

    EncodeTiledFn fn = encode_fn();
    if (!fn) return (int)cudaErrorNotSupported;
    // K as rows of a token's 128 codes, V as rows of a dimension's bt codes; a
    // block of a head is one box, swizzled over its row length
    CUtensorMap kmap, vmap;
    auto encode = [&](CUtensorMap *m, const uint8_t *pool, int width, int height, CUtensorMapSwizzle swz) {
        const cuuint64_t dims[2] = {(cuuint64_t)width, (cuuint64_t)a.n_blocks * a.H * height};
        const cuuint64_t strides[1] = {(cuuint64_t)width};
        const cuuint32_t box[2] = {(cuuint32_t)width, (cuuint32_t)height}, es[2] = {1, 1};
        return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t *>(pool), dims, strides, box, es,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, swz, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    };
    if (!encode(&kmap, a.kc, kD, a.bt, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode(&vmap, a.vc, a.bt, kD,
                a.bt == 32   ? CU_TENSOR_MAP_SWIZZLE_32B
                : a.bt == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                             : CU_TENSOR_MAP_SWIZZLE_128B))
        return (int)cudaErrorInvalidValue;
    // Columns of a segment: the least shape that holds an average request's rows
    // and one row's heads.  One row of 5 heads behind 131072 tokens takes 55.7 us
    // with 16 columns, 56.0 with 48 and 71 with 80 (behind 200: 11.3, 12.3, 12.3);
    // 8 rows of 5 heads to a request 198 us with 48, 237 with 80 and 348 with 16;
    // 32 rows of 5 heads 60 us with 80, 71.5 with 48 and 118 with 16.
    const int64_t avg = (int64_t)((a.R + a.n_req - 1) / a.n_req) * p.G;
    p.cols = avg <= 16 ? 16 : avg <= 48 ? 48 : 80;
    p.fit = p.cols / p.G;
    const cudaError_t e = p.cols == 16   ? launch_ctx<16>(kmap, vmap, p, st)
                          : p.cols == 48 ? launch_ctx<48>(kmap, vmap, p, st)
                                         : launch_ctx<80>(kmap, vmap, p, st);
    if (e != cudaSuccess) return (int)e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)a.R, (unsigned)a.H);
    cfg.blockDim = dim3((unsigned)std::min(p.G, kJoinWarps) * 32);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return (int)cudaLaunchKernelEx(&cfg, k_attn_join, p);
}

}  // namespace w12i
