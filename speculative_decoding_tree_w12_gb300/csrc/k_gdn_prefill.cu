// Recurrent (Gated DeltaNet) layer over whole prompts (sm_103a).
//
// A head's state S (d_v x d_k) follows S <- a S (I - b k k^T) + b v k^T, and a
// token's output is o = S q of the new state.  64 tokens are taken at once.
// With G_i the product of the gates from the chunk's start to token i and D_ij
// that of the gates j + 1 .. i, the vectors u_i = b_i (v_i - a_i S_{i-1} k_i)
// solve
//     (I + L) U = X,   L_ij = b_i D_ij k_i.k_j (j < i),   x_i = b_i (v_i - G_i S k_i),
// with S the state in front of the chunk, and
//     o_i = G_i S q_i + sum over j <= i of A_ij u_j,   A_ij = D_ij q_i.k_j,
//     S'  = G_C S + sum over j of D_Cj u_j k_j^T.
// M = (I + L)^-1 and A need no state, so they are made a chunk ahead.  The D_ij
// are running products, never quotients: a gate of zero forgets, as it should.
//
// A CTA takes one (request, head) after another; the state rows c lie on the 128 lanes of tensor memory throughout, so that
// all its products take their left operand from there and no operand but M and A is ever written to shared memory:
//     D_K[c][j] = S k_j    D_Q[c][j] = S q_j    U[c][i] = X M^T    U A^T    S' = U K.
// An FP32 operand (S, U, X, M, A) is three BF16 pieces that add up to it exactly: two (2^-17) would be the largest error of the
// layer by far, and F16 pieces need a unit, under which small values are lost beside large ones (a row's 64 tokens differ by what
// their gates forget or raise).  Keys and queries are BF16 as they are; of two FP32 operands' nine pairs of pieces (X M^T, U A^T) the
// three smallest are left out: 2^-21 of a product at most, 2^-24 in the mean.  All accumulation is FP32.
//
// A chunk runs through S's pieces -> S k -> X -> U -> U's pieces -> U K -> S', each step of which waits for the one before
// it; the rest (A, M, U A^T and the outputs) is other warps' work, a chunk ahead or beside it:
//  * state warps (0..7; two threads to a state row): S, which stays in their registers, and U scaled for S',
//  * token warps (8..15; two threads to a state row): X, U for A, and the outputs,
//  * gate warps (16..19; a thread to a row of k.k or q.k): the gates' products, L with the inverses of its four diagonal
//    blocks of 16, whose columns are solved in registers, and A,
//  * inverse warps (20..23): M, the blocks below those from them,
//  * warp 24 issues the products with the state, warp 25 the copies by TMA, warps 26 and 27 make M's pieces.
// A chunk takes 4.2 to 4.4 us (8,000 to 8,600 cycles) however many there are: sixteen prompts of up to 8192 tokens x 32 heads
// 1425 us, 2.5 times what their bytes take at the measured copy bandwidth.  That is the way through the steps above, each with its
// hand-over to the next one's warps, on a full machine: S's pieces 1,900 cycles (three BF16 pieces take 11 cycles of a scheduler for
// two values of 32 lanes), what of S k is left then and X 2,000, M X 1,250, U's pieces 1,500, U K 700, S' 850.  The schedulers
// issue in 55 % of the cycles, the tensor cores work in 37 %.
// Most products are issued in rolled loops and the code is kept short: straight-line code of a few times this length spent half
// its time on its own way in.  A new pair costs 2.0 us more than its chunks, 4.2 where a state is read.
// Every wait is bounded; when one has run out no state that what did not come is part of is written.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstddef>
#include <vector>

#include "w12_device.cuh"

using namespace w12d;

namespace {

constexpr int kD = 128;             // head dimension
constexpr int kC = 64;              // tokens of a chunk
constexpr int kThreads = 32 * 28;
// the roles' first threads, and their registers (the launch's where they are equal to it)
constexpr int kToken0 = 256, kGate0 = 512, kInv0 = 640, kIssue0 = 768;
constexpr int kRegsLaunch = 72, kRegsState = 104, kRegsGate = 56, kRegsInv = 56, kRegsIssue = 40;
static_assert(256 * (kRegsState + kRegsLaunch) + 128 * (kRegsGate + kRegsInv + kRegsIssue) <= kThreads * kRegsLaunch, "register shares");

// tensor memory columns: all 512 are one CTA's, from column 0 on
constexpr uint32_t kColS = 0;       // S: three pieces of 64 columns; then three of U for S', 32 each,
constexpr uint32_t kColUA = 96;     // and three of U for A, by token_piece
constexpr uint32_t kColDQ = 192;    // S q
constexpr uint32_t kColDK = 256;    // S k; then, with the next 64 columns, U K
constexpr uint32_t kColX = 256;     // X's three pieces, by token_piece: a thread's lie over the S k that it alone has read
constexpr uint32_t kColU = 384;     // U; then, when its pieces have been made, U A
constexpr uint32_t kColKK = 448;    // k.k (lanes 0..63) and q.k (lanes 64..127) of the next chunk

// where 32 tokens' (half 0 or 1) high, middle and low pieces (0 .. 2) are, 16 columns each: the first two beside one another
__host__ __device__ constexpr uint32_t token_piece(int piece, int half) { return piece < 2 ? 32 * half + 16 * piece : 64 + 16 * half; }

// A piece of M or A in shared memory, rows of 32 BF16 under the 64-byte swizzle: all rows' first half, then the lower rows' second
// (the upper rows have none)
constexpr int kTriBytes = (kC + kC / 2) * 64, kTriRight = kC * 64;
__host__ __device__ constexpr int tri_at(int row, int col)
{
    return (col < 32 ? row * 64 : kTriRight + (row - 32) * 64) + ((((col & 31) >> 3) ^ ((row >> 1) & 3)) << 4);
}

// L, then M: three blocks of 32 x 32 (the one above the diagonal is zero), their FP32 rows 16-byte aligned and 4 banks apart
constexpr int kLS = 36;
constexpr int kL11 = 0, kL22 = 32 * kLS, kL21 = 2 * 32 * kLS, kLFloats = 3 * 32 * kLS;
constexpr int kBarGate = 1, kBarInv = 2, kBarState = 3;   // named barriers: of the gate warps, the inverse warps, the state warps
constexpr int kStages = 3;          // of keys and queries (their chunk is prepared while two others are in use)

// what a chunk is of
enum Start : int32_t { kGoesOn, kFromState, kFromZero, kFromOne };
struct Chunk {
    const float *from;              // the state in front, where one is loaded
    float *to;                      // where the state behind it goes, or null
    int32_t row0, n;                // first row, rows
    int32_t out;                    // rows whose outputs are wanted: all of them or none
    int32_t h;
    Start start;                    // where the state in front comes from
};
constexpr int kChunks = 8;          // descriptions kept

struct PrefillShared {
    uint8_t KQ[kStages][2 * 128 * 128];   // [stage][feature half][key rows, query rows][64 BF16], 128-byte swizzle
    uint8_t A[2][3][kTriBytes];     // pieces of A and M
    uint8_t M[3][kTriBytes];
    uint16_t V[2][kC * kD];
    alignas(16) float L[2][kLFloats];   // then, in place, M
    alignas(16) float T[32 * kLS];      // products in between
    alignas(16) float next[kC];     // the gates of tokens 1 .. 63, then 1
    alignas(16) float b[4][kC];     // of chunk c in [c % 4]: strengths, -b_i G_i, G_i, D_Ci
    alignas(16) float bG[4][kC];
    alignas(16) float G[4][kC];
    alignas(16) float tail[4][kC];
    float gates[2];                 // products of the gates of tokens 0 .. 31 and 32 .. 63
    Chunk chunk[kChunks];           // of chunk c in [c % 8], by the thread that issues the copies
    unsigned long long told[4];                         // it is there
    unsigned long long full[kStages], empty[kStages];   // keys and queries
    unsigned long long vfull[2], vempty[2];             // values
    unsigned long long gready[2], gused[2];             // A and the gates' products are there; A has been read
    unsigned long long lready[2], inverted[2], lfree[2];   // L is there, M in its place, M taken from there
    unsigned long long mready[2];                       // M is there (two barriers for one M: a waiter may be a phase late)
    unsigned long long bar_kk;
    unsigned long long have_s[2], have_us[2], have_x, have_u;   // operands written (S and U for S' by halves)
    unsigned long long read_o;                          // the outputs have been read
    unsigned long long done_k, done_u, done_s, done_o;  // products done
    unsigned long long last, last_kk;
    uint32_t tmem;
    int32_t abort;
    int32_t total;                  // chunks of this CTA
    int32_t silent;                 // whose outputs nobody wants (Q and P)
    uint16_t order[w12i::kMaxBudget];   // the requests, those with the most rows first
};
static_assert(offsetof(PrefillShared, L) % 16 == 0 && kLFloats % 4 == 0, "rows of four floats");
static_assert(offsetof(PrefillShared, T) == offsetof(PrefillShared, L) + sizeof(PrefillShared::L), "T behind L");
static_assert(sizeof(PrefillShared) + 1024 <= 227 * 1024, "shared memory above the per-CTA limit");
static_assert(offsetof(PrefillShared, M) % 1024 == 0 && offsetof(PrefillShared, A) % 1024 == 0, "swizzled tiles");
static_assert(offsetof(PrefillShared, V) % 128 == 0 && offsetof(PrefillShared, full) % 8 == 0, "copies and barriers");
constexpr uint32_t kKqBytes = sizeof(PrefillShared::KQ) / kStages, kVBytes = sizeof(PrefillShared::V) / 2;

// Few long requests leave most SMs without one.  The state behind a part of a request is S P + Q in that in front: Q what the
// part makes of a state of zero, P what it makes of the unit matrix without values.  So each is cut into n = (j + 1) w + 1 like
// pieces, and two launches run them, one CTA to an item:
//  * kAhead: the first w pieces as they are, and Q and P of the j segments of w pieces behind them, noted after every piece,
//  * k_gdn_join: the states in front of every piece but the first w from those,
//  * kPieces: those pieces, now with their outputs.
// That takes w + 1 pieces' time of n, and (2 j + 1) and (j w + 1) CTAs a pair (one of 4096 tokens, 4 heads: 278 us in one
// part a head, 83 cut; of 32768 tokens, 32 heads: 2207 and 1258).  The launches overlap: each begins where SMs are left, and waits for the
// one before it only for what that wrote.
enum Mode : int32_t { kWhole, kAhead, kPieces };

struct SplitParams {
    Mode mode;
    int32_t j, w;                   // at most; pieces of a segment
    float *states;                  // [pair][j w + 1][Q or the state in front, P][kD][kD]
    int32_t *failed;                // [pair][2 j + 1]: whether an item of kAhead has given up
};

// Segments of a request of nc chunks.  The join takes a product of 1.1 us for each piece of them, so no more than pay for
// theirs; and it and one more launch some 30 us, seven chunks' time, which the j w pieces that run beside the others have to
// save.  (One request of 32 heads, j = 1: 14 chunks 71 us whole, 76 cut, 16 chunks 79 and 80, 20 chunks 96 and 92; of 16 heads: 8
// chunks 45 and 50, 10 chunks 54 and 54, 12 chunks 62 and 61.)
__host__ __device__ inline int split_segments(int nc, int j, int w)
{
    while (j > 0 && (j * j > 2 * nc || (j + 1) * w + 1 > nc)) --j;
    return (int64_t)nc * j * w < 7 * ((j + 1) * w + 1) ? 0 : j;
}

struct PrefillParams {
    const float *S0;                // may be null: zero
    float *state, *o;
    const float *alpha, *beta;
    const int32_t *off;
    int32_t H, group, n_req, n_rows;
    SplitParams split;
    uint32_t subs, items;           // items of a pair; n_req * H of them each
    uint32_t polls;                 // of a wait, before it gives up
    int32_t *status;
    int32_t debug_flags;            // test hooks, bit 0: CTA 0 announces its first copies and leaves them out; bit 5: its token
                                    // warps' budget ends at its last chunk's S k
};

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

// D[tmem] (+)= A[smem] * B[smem]
__device__ __forceinline__ void tc_mma_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ bool elect_lane()
{
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
    return e != 0;
}

// Matrix descriptors from their lower word (address and leading offset): rows of 64 values under the 128-byte swizzle, eight
// rows 1024 bytes on.  desc_k: the rows are the operand's own; desc_mn: they are its K index, the next 64 values
// 128 rows of 128 bytes further on.
__device__ __forceinline__ uint32_t desc_low(uint32_t saddr) { return (saddr >> 4) & 0x3FFFu; }
__device__ __forceinline__ uint64_t desc_of(uint32_t low)
{
    constexpr uint32_t high = (1024u >> 4) | (1u << 14) | (2u << 29);   // stride, version 1, swizzle
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(low), "n"(high));
    return d;
}
__device__ __forceinline__ uint64_t desc_k(uint32_t low) { return desc_of(low | (1u << 16)); }
// ... rows of 32 values under the 64-byte swizzle, eight rows 512 bytes on
__device__ __forceinline__ uint64_t desc_tri(uint32_t low)
{
    constexpr uint32_t high = (512u >> 4) | (1u << 14) | (4u << 29);
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(low | (1u << 16)), "n"(high));
    return d;
}
__device__ __forceinline__ uint64_t desc_mn(uint32_t low) { return desc_of(low | ((128u * 128u / 16u) << 16)); }

constexpr uint32_t kBMnMajor = 1u << 16;   // instruction descriptor: B's rows are its K index

// The high, middle and low BF16 pieces of 2N values, N words each: `put(piece, words)`.  Every piece is
// the upper half of what the ones before it left, so the three add up exactly.
template <int N, class F>
__device__ __forceinline__ void pieces3(float (&x)[2 * N], F put)
{
#pragma unroll
    for (int piece = 0; piece < 3; ++piece) {
        uint32_t w[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            w[i] = __byte_perm(__float_as_uint(x[2 * i]), __float_as_uint(x[2 * i + 1]), 0x7632);
            if (piece < 2) {
                // (the shift runs beside the logic operations, so taking both halves from the word is a fifth faster)
                const float2 r = __ffma2_rn(make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u)),
                                            make_float2(-1.f, -1.f), make_float2(x[2 * i], x[2 * i + 1]));
                x[2 * i] = r.x;
                x[2 * i + 1] = r.y;
            }
        }
        put(piece, w);
    }
}

__device__ __forceinline__ void tmem_st_x8(uint32_t taddr, const uint32_t (&r)[8])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

// 32 lanes x N columns as floats (complete after tmem_ld_wait)
template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, float (&x)[N])
{
#pragma unroll
    for (int i = 0; i < N; i += 16)
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
            "%15}, [%16];"
            : "=f"(x[i]), "=f"(x[i + 1]), "=f"(x[i + 2]), "=f"(x[i + 3]), "=f"(x[i + 4]), "=f"(x[i + 5]), "=f"(x[i + 6]),
              "=f"(x[i + 7]), "=f"(x[i + 8]), "=f"(x[i + 9]), "=f"(x[i + 10]), "=f"(x[i + 11]), "=f"(x[i + 12]),
              "=f"(x[i + 13]), "=f"(x[i + 14]), "=f"(x[i + 15])
            : "r"(taddr + i)
            : "memory");
}

// N values of shared memory, the same ones for every lane
template <int N>
__device__ __forceinline__ void read_n(const float *src, float (&x)[N])
{
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
        const float4 v = reinterpret_cast<const float4 *>(src)[i];
        x[4 * i] = v.x;
        x[4 * i + 1] = v.y;
        x[4 * i + 2] = v.z;
        x[4 * i + 3] = v.w;
    }
}

// eight values of global memory, a whole 32-byte sector a lane (half of one at a time, as four values are, takes the load and store
// units twice as long where every lane has a row of its own)
__device__ __forceinline__ void load8(const float *src, float *x)
{
    asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]), "=f"(x[4]), "=f"(x[5]), "=f"(x[6]), "=f"(x[7])
                 : "l"(src)
                 : "memory");
}
__device__ __forceinline__ void store8(float *dst, const float *x)
{
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]),
                 "f"(x[5]), "f"(x[6]), "f"(x[7])
                 : "memory");
}

// x *= y, two at a time
template <int N>
__device__ __forceinline__ void mul_n(float (&x)[N], const float (&y)[N])
{
#pragma unroll
    for (int i = 0; i < N; i += 2) {
        const float2 r = __fmul2_rn(make_float2(x[i], x[i + 1]), make_float2(y[i], y[i + 1]));
        x[i] = r.x;
        x[i + 1] = r.y;
    }
}
// this warp's tensor-memory accesses are done: one arrival for the warp
__device__ __forceinline__ void warp_arrive(uint32_t bar, int lane)
{
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
}

// A thread's bounded waits, in few instructions (there are three dozen of them): `left` is what it may still poll in all its
// waits together (the time limit and 16 polls for every chunk), a poll sleeping up to kWaitSleepNs.  When that has run out no wait
// lasts any more, so every role runs to its end.  What is made of what did not come is marked before it is signalled, so nothing
// that it is part of is stored.  What is read on the way may be old or half written: so no address is made of it that is not checked
// where it is used.  (Marked at once, in every wait: sixteen prompts of up to 1024 tokens x 32 heads 201 us, 190 so.)
struct Waits {
    uint32_t left;

    __device__ __forceinline__ bool on(unsigned long long &bar, uint32_t parity)
    {
        const uint32_t at = smem_u32(&bar);
#pragma unroll 1
        while (!mbar_try_wait_sleep(at, parity, kWaitSleepNs)) {
            if (left == 0) return false;
            --left;
        }
        return true;
    }

    // in front of a signal to another role, and at a role's end
    __device__ __forceinline__ void mark(PrefillShared &s) const
    {
        if (left == 0) *(volatile int32_t *)&s.abort = 1;
    }
};

// whether `ok` holds in every one of so many threads, the same answer in all of them
__device__ __forceinline__ bool all_of(int id, int threads, bool ok)
{
    uint32_t all;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %3, 0;\n\tbarrier.cta.red.and.pred q, %1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(all)
                 : "r"(id), "r"(threads), "r"((uint32_t)ok)
                 : "memory");
    return all != 0;
}

// a wait of its own: for what is in flight at the end
__device__ __forceinline__ void drain(unsigned long long &bar, uint32_t parity, const PrefillParams &p)
{
    uint32_t left = p.polls;
#pragma unroll 1
    while (!mbar_try_wait_sleep(smem_u32(&bar), parity, kWaitSleepNs) && --left) {
    }
}

// a request's rows, or -1 where its offsets make no sense
__device__ __forceinline__ int request_rows(const PrefillParams &p, int r)
{
    const int o0 = p.off[r], o1 = p.off[r + 1];
    return o0 < 0 || o1 < o0 || o1 > p.n_rows ? -1 : o1 - o0;
}

// The (request, head) pairs of this CTA, one after another: the requests by their rows, the heads of one request beside one
// another, dealt out to the CTAs forth and back, so that each gets a like share of long and short ones.  The rings count
// the CTA's chunks through all of them.
__device__ __forceinline__ uint32_t item(uint32_t cycle)
{
    return cycle * gridDim.x + (cycle & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
}

__device__ __forceinline__ int chunks_of(int rows) { return rows > 0 ? (rows - 1) / kC + 1 : 0; }

// the chunks of item `sub` of a request of nc of them
struct Part {
    int first, end;
    int j;                          // the request's segments
    int slot;                       // kAhead: of the first state that is noted; kPieces: of the one in front
};
__device__ __forceinline__ int piece_start(const PrefillParams &p, int nc, int j, uint32_t i)
{
    // In eighths of a piece: the first w pieces are shorter by one, since a chunk with its outputs takes longer than one of Q's or P's (one
    // request of 32768 tokens, 32 heads: 1316 us with like pieces, 1258 so, 1329 with two eighths).
    const uint32_t w = p.split.w, n = 8 * (j * w + 1) + 7 * w, like = (uint32_t)nc / n, at = i < w ? 7 * i : 8 * i - w;
    return (int)(at * like + at * (nc - n * like) / n);
}
__device__ __forceinline__ Part part_of(const PrefillParams &p, int nc, int sub)
{
    if (p.split.mode == kWhole) return Part{0, nc, 0, 0};
    const int j = split_segments(nc, p.split.j, p.split.w), w = p.split.w;
    if (p.split.mode == kAhead) {
        const int seg = (sub + 1) >> 1;
        if (seg == 0) return Part{0, j ? piece_start(p, nc, j, w) : nc, j, 0};
        if (seg > j) return Part{0, 0, j, 0};
        return Part{piece_start(p, nc, j, seg * w), piece_start(p, nc, j, (seg + 1) * w), j, (seg - 1) * w + 1};
    }
    if (j == 0 || sub > j * w) return Part{0, 0, j, 0};
    return Part{piece_start(p, nc, j, w + sub), piece_start(p, nc, j, w + sub + 1), j, sub};
}
// the state (or Q) in front of piece w + slot, P with `which` 1
__device__ __forceinline__ float *split_state(const SplitParams &s, int pair, int slot, int which)
{
    return s.states + (((size_t)pair * (s.j * s.w + 1) + slot) * 2 + which) * (kD * kD);
}

// ---------------------------------------------------------------------------
// state warps
// ---------------------------------------------------------------------------

__device__ __forceinline__ void state_warps(const PrefillParams &p, PrefillShared &s)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, part = warp >> 2;
    const int c = (warp & 3) * 32 + lane;                                 // state row
    const uint32_t tm = (uint32_t)((warp & 3) * 32) << 16;                // this warp's lanes
    Waits waits{p.polls + 16u * s.total};
    auto wait = [&](unsigned long long &bar, uint32_t parity) {
        waits.on(bar, parity);
        tc_fence_after();
    };
    const int total = s.total;
    if (p.split.mode == kPieces) {
        pdl_wait();                               // the states in front come from the launches before
        const uint32_t a_rank = p.subs * p.H, pair = s.order[blockIdx.x / a_rank] * p.H + blockIdx.x % a_rank % p.H;
        const int all = 2 * p.split.j + 1;
        int failed = 0;
#pragma unroll 1
        for (int e = lane; e < all; e += 32) failed |= __ldcg(p.split.failed + pair * all + e);
        if (__any_sync(0xffffffffu, failed)) waits.left = 0;   // (nothing is made of what did not come about)
    }
    float S[64];
#pragma unroll 1
    for (int g = 0; g < total; ++g) {
        wait(s.told[g & 3], (g >> 2) & 1);
        const Chunk &t = s.chunk[g % kChunks];
        const int at = c * kD + 64 * part;                                // this thread's half of the row
        if (t.start != kGoesOn) {
            const float *from = *(const float *const volatile *)&t.from;   // (null behind a wait that has run out, maybe)
            if (t.start == kFromState && from) {
#pragma unroll
                for (int i = 0; i < 64; i += 8) load8(from + at + i, S + i);
            } else {
#pragma unroll
                for (int i = 0; i < 64; ++i) S[i] = 0.f;
            }
            if (t.start == kFromOne) {
#pragma unroll
                for (int i = 0; i < 64; ++i) S[i] = 64 * part + i == c ? 1.f : 0.f;
            }
        }
        const int k4 = g & 3;
        const uint32_t par = g & 1, par2 = (g >> 1) & 1;
        // S's pieces, a half of this thread's features at a time (over the last chunk's U, which A has been multiplied by)
        if (g > 0) wait(s.done_o, par ^ 1u);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            float z[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) z[i] = S[16 * q + i];
            pieces3<8>(z, [&](int piece, const uint32_t (&w)[8]) { tmem_st_x8(tm + kColS + 64 * piece + 32 * part + 8 * q, w); });
            if (q & 1) {
                tmem_st_wait();
                warp_arrive(smem_u32(&s.have_s[q >> 1]), lane);
            }
        }

        // U scaled for S', over S's pieces (which have been read: S q came before U)
        wait(s.gready[g & 1], par2);
        wait(s.done_u, par);
#pragma unroll 1
        for (int q = 0; q < 2; ++q) {
            const int t0 = 32 * part + 16 * q;
            float x[16], f[16];
            tmem_ld<16>(tm + kColU + t0, x);
            read_n(s.tail[k4] + t0, f);
            tmem_ld_wait();
            mul_n(x, f);
            pieces3<8>(x, [&](int piece, const uint32_t (&w)[8]) { tmem_st_x8(tm + kColS + 32 * piece + t0 / 2, w); });
            tmem_st_wait();
            warp_arrive(smem_u32(&s.have_us[q]), lane);
        }

        // S' = G_C S + U K
        const float gc = s.G[k4][kC - 1];
        bool good = true;
        wait(s.done_s, par);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            float z[32];
            tmem_ld<32>(tm + kColDK + 64 * part + 32 * q, z);
            // Whether a wait has run out for what this state is made of: one answer for all its rows, given in every chunk (where
            // there is a state to write is no longer the same to all of them when one of their own has run out).
            if (q == 0) good = all_of(kBarState, 256, waits.left && !*(volatile int32_t *)&s.abort);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
                const float2 n = __ffma2_rn(make_float2(gc, gc), make_float2(S[32 * q + i], S[32 * q + i + 1]), make_float2(z[i], z[i + 1]));
                S[32 * q + i] = n.x;
                S[32 * q + i + 1] = n.y;
            }
        }
        if (good && t.to) {
#pragma unroll
            for (int i = 0; i < 64; i += 8) store8(t.to + at + i, S + i);
        }
    }
    waits.mark(s);
}

// ---------------------------------------------------------------------------
// token warps
// ---------------------------------------------------------------------------

__device__ __forceinline__ void token_warps(const PrefillParams &p, PrefillShared &s)
{
    const int lane = threadIdx.x & 31, warp = (threadIdx.x - kToken0) >> 5, part = warp >> 2;
    const int c = (warp & 3) * 32 + lane, t0 = 32 * part;                 // state row, first token
    const uint32_t tm = (uint32_t)((warp & 3) * 32) << 16;
    Waits waits{p.polls + 16u * s.total};
    auto wait = [&](unsigned long long &bar, uint32_t parity) {
        waits.on(bar, parity);
        tc_fence_after();
    };
    // the pieces of 16 tokens' values, from the first or the second of this thread's sixteens
    auto put = [&](uint32_t col, int sixteen, float (&z)[16]) {
        pieces3<8>(z, [&](int piece, const uint32_t (&w)[8]) { tmem_st_x8(tm + col + token_piece(piece, part) + 8 * sixteen, w); });
    };
    const int total = s.total;
    const int impatient = (p.debug_flags & 32) && blockIdx.x == 0 && p.split.mode != kPieces ? total - 1 : -1;   // (test hook)
#pragma unroll 1
    for (int g = 0; g < total; ++g) {
        const int st = g & 1, k4 = g & 3;
        const uint32_t par = g & 1, par2 = (g >> 1) & 1;
        // X = b (v - G S k); b v while S k is being made
        wait(s.vfull[st], par2);
        wait(s.gready[st], par2);
        float x[32];
#pragma unroll
        for (int q = 0; q < 32; q += 8) {
            float e[8];
            const uint16_t *v = s.V[st] + (t0 + q) * kD + c;
            read_n(s.b[k4] + t0 + q, e);
#pragma unroll
            for (int j = 0; j < 8; ++j) x[q + j] = e[j] * __uint_as_float((uint32_t)v[j * kD] << 16);
        }
        // (What has been read here and what a copy writes here next meet in different ways to memory, which neither the order of the
        // program nor the arrival's own keeps apart.)
        __syncwarp();
        if (lane == 0) {
            fence_async_shared();
            mbar_arrive(smem_u32(&s.vempty[st]));
        }
        wait(s.done_k, par);
        if (g == impatient) waits.left = 0;
#pragma unroll
        for (int q = 0; q < 32; q += 16) {
            float d[16], f[16];
            tmem_ld<16>(tm + kColDK + t0 + q, d);
            read_n(s.bG[k4] + t0 + q, f);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 16; j += 2) {
                const float2 r = __ffma2_rn(make_float2(f[j], f[j + 1]), make_float2(d[j], d[j + 1]), make_float2(x[q + j], x[q + j + 1]));
                x[q + j] = r.x;
                x[q + j + 1] = r.y;
            }
        }
#pragma unroll
        for (int q = 0; q < 32; q += 16) {
            float z[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) z[j] = x[q + j];
            put(kColX, q >> 4, z);
        }
        tmem_st_wait();
        waits.mark(s);
        warp_arrive(smem_u32(&s.have_x), lane);
        if (s.silent) continue;

        // U's pieces for A, over S's (S q is there)
        wait(s.done_u, par);
#pragma unroll 1
        for (int q = 0; q < 2; ++q) {
            float z[16];
            tmem_ld<16>(tm + kColU + t0 + 16 * q, z);
            tmem_ld_wait();
            put(kColUA, q, z);
        }
        tmem_st_wait();
        warp_arrive(smem_u32(&s.have_u), lane);

        // o = G S q + U A.  U A has an accumulator of its own: its additions round at its own size then, not at that of S q (error of
        // the outputs against 64 bits with gates near 1 6.4e-7 on top of S q, 3.5e-7 so; sixteen prompts of up to 4096 tokens x 32
        // heads 723 us and 730).
        wait(s.done_o, par);
        const size_t step = (size_t)p.H * kD;
        const Chunk &t = s.chunk[g % kChunks];
        float *dst = p.o + ((size_t)(t.row0 + t0) * p.H + t.h) * kD + c;
        int left = min(t.out, p.n_rows - t.row0) - t0;
#pragma unroll
        for (int q = t0; q < t0 + 32; q += 16, left -= 16) {
            float z[16], f[16], x[16];
            tmem_ld<16>(tm + kColDQ + q, z);
            tmem_ld<16>(tm + kColU + q, x);
            read_n(s.G[k4] + q, f);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 16; j += 2) {
                const float2 r = __ffma2_rn(make_float2(f[j], f[j + 1]), make_float2(z[j], z[j + 1]), make_float2(x[j], x[j + 1]));
                x[j] = r.x;
                x[j + 1] = r.y;
            }
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                if (j < left) *dst = x[j];
                dst += step;
            }
        }
        warp_arrive(smem_u32(&s.read_o), lane);
    }
    waits.mark(s);
}

// ---------------------------------------------------------------------------
// gate warps
// ---------------------------------------------------------------------------

// the pieces of 16 values into row `row` of tiles, from column `col0` on (a multiple of 16)
__device__ __forceinline__ void put_row(uint8_t (&tile)[3][kTriBytes], int row, int col0, float (&x)[16])
{
    pieces3<8>(x, [&](int piece, const uint32_t (&w)[8]) {
#pragma unroll
        for (int q = 0; q < 2; ++q)
            *reinterpret_cast<uint4 *>(tile[piece] + tri_at(row, col0 + 8 * q)) = make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
    });
}

// Two lower-triangular 16 x 16 blocks with ones on their diagonals, one below the other's corner, inverted in place by one
// warp, a column to a lane and four rows at a time: x_i = [i = j] - sum over l < i of L_il x_l.  A lane reads back only
// what it wrote itself.
__device__ __forceinline__ void invert16(float *L, int lane)
{
    float *B = L + (lane >> 4) * 16 * (kLS + 1);
    const int col = lane & 15;
#pragma unroll 1
    for (int r0 = 0; r0 < 16; r0 += 4) {
        float *R = B + r0 * kLS;
        float x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = r0 + i == col ? 1.f : 0.f;
#pragma unroll 1
        for (int l = 0; l < r0; l += 4) {
            float y[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) y[e] = B[(l + e) * kLS + col];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float4 v = *reinterpret_cast<const float4 *>(R + i * kLS + l);
                x[i] = fmaf(-v.x, y[0], fmaf(-v.y, y[1], fmaf(-v.z, y[2], fmaf(-v.w, y[3], x[i]))));
            }
        }
        const float l10 = R[kLS + r0];
        const float2 l2 = *reinterpret_cast<const float2 *>(R + 2 * kLS + r0);
        const float4 l3 = *reinterpret_cast<const float4 *>(R + 3 * kLS + r0);
        x[1] = fmaf(-l10, x[0], x[1]);
        x[2] = fmaf(-l2.x, x[0], fmaf(-l2.y, x[1], x[2]));
        x[3] = fmaf(-l3.x, x[0], fmaf(-l3.y, x[1], fmaf(-l3.z, x[2], x[3])));
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i) R[i * kLS + col] = x[i];
    }
}

__device__ __forceinline__ void gate_warps(const PrefillParams &p, PrefillShared &s)
{
    const int tid = threadIdx.x - kGate0, lane = tid & 31, warp = tid >> 5;
    const int i = tid & 63;                       // token of the chunk
    const bool query = warp >= 2;                 // this thread's row: k_i.k or q_i.k
    Waits waits{p.polls + 16u * s.total};
    const int blocks = (warp & 1) ? 4 : 2;        // of 16 columns that its warp's rows reach into
    const uint32_t tm = (uint32_t)(warp * 32) << 16;
    // warp 3: k.k and q.k of a chunk whose rows have arrived.  Rows behind the request's end are another
    // request's, or none: whatever they hold becomes zero.
    auto products = [&](int g, int valid) {
        const int st = g % kStages;
        waits.on(s.full[st], (g / kStages) & 1);
        __syncwarp();
        if (valid < kC) {
            waits.on(s.vfull[g & 1], (g >> 1) & 1);
            __syncwarp();
#pragma unroll 1
            for (int e = lane; e < (kC - valid) * 16; e += 32) {
                const int row = valid + (e >> 4), q = e & 15;
                const uint4 z = make_uint4(0, 0, 0, 0);
                uint8_t *half = s.KQ[st] + (q >> 3) * (128 * 128);
                *reinterpret_cast<uint4 *>(half + row * 128 + (q & 7) * 16) = z;
                *reinterpret_cast<uint4 *>(half + (kC + row) * 128 + (q & 7) * 16) = z;
                *reinterpret_cast<uint4 *>(s.V[g & 1] + row * kD + q * 8) = z;
            }
            fence_async_shared();
            __syncwarp();
        }
        tc_fence_after();
        const uint32_t kq = smem_u32(s.KQ[st]);
        if (elect_lane()) {
#pragma unroll 1
            for (int half = 0; half < 2; ++half) {
                const uint32_t x = desc_low(kq + half * 128 * 128);
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                    tc_mma_ss(kColKK, desc_k(x + ks * 2), desc_k(x + ks * 2), idesc_bf16_f32(128, kC), (uint32_t)(half | ks));
            }
            tc_commit(smem_u32(&s.bar_kk));
        }
        __syncwarp();
    };
    // the next chunk: the gate and the strength of this thread's token (1 and 0 behind the end), its rows
    int valid = 0;
    float a = 1.f, b = 0.f;
    auto fetch = [&](int g) {
        waits.on(s.told[g & 3], (g >> 2) & 1);
        const Chunk &t = s.chunk[g % kChunks];
        const size_t at = (size_t)(t.row0 + i) * p.H + t.h;
        valid = min(t.n, p.n_rows - t.row0);      // (less only behind a wait that has run out)
        a = i < valid ? p.alpha[at] : 1.f;
        b = i < valid ? p.beta[at] : 0.f;
    };
    const int total = s.total;
    if (total > 0) fetch(0);
#pragma unroll 1
    for (int g = 0; g < total; ++g) {
        const int st = g & 1, k4 = g & 3;
        const uint32_t par2 = (g >> 1) & 1;
        if (warp == 3) products(g, valid);
        const float strength = b;
        float up = a, down = a;
        if (!query) {
            // products of the gates from this block of 32 tokens' start to token i, and from behind it to the block's end
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const float u = __shfl_up_sync(0xffffffffu, up, o), v = __shfl_down_sync(0xffffffffu, down, o);
                if (lane >= o) up *= u;
                if (lane + o < 32) down *= v;
            }
            down = __shfl_down_sync(0xffffffffu, down, 1);
            if (lane == 31) down = 1.f;
            s.next[(i + kC - 1) & (kC - 1)] = i ? a : 1.f;
            if (lane == 31) s.gates[warp] = up;
        }
        named_bar(kBarGate, 128);
        if (g + 1 < total) fetch(g + 1);
        if (!query) {
            const float G = i < 32 ? up : up * s.gates[0];
            s.b[k4][i] = strength;
            s.G[k4][i] = G;
            s.bG[k4][i] = -strength * G;
            s.tail[k4][i] = i < 32 ? down * s.gates[1] : down;
        }
        waits.on(s.bar_kk, g & 1);
        tc_fence_after();
        // D_ij (for L times b_i), from j = i down, times the row of k.k or q.k
        {
            float d = query ? 1.f : strength;
            if (g >= 2) waits.on(query ? s.gused[st] : s.lfree[st], par2 ^ 1u);
            const int last = query ? i : i - 1;   // the row's last entry
#pragma unroll 1
            for (int J = blocks - 1; J >= 0; --J) {
                float x[16], f[16];
                tmem_ld<16>(tm + kColKK + 16 * J, x);
                read_n(s.next + 16 * J, f);
                tmem_ld_wait();
                if (J >= blocks - 2) {            // columns among which this warp's diagonals lie
#pragma unroll
                    for (int j = 15; j >= 0; --j) {
                        d *= 16 * J + j < i ? f[j] : 1.f;
                        x[j] = 16 * J + j <= last ? x[j] * d : 0.f;
                    }
                } else {
#pragma unroll
                    for (int j = 15; j >= 0; --j) {
                        d *= f[j];
                        x[j] *= d;
                    }
                }
                if (query) {
                    put_row(s.A[st], i, 16 * J, x);
                } else {
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        *reinterpret_cast<float4 *>(s.L[st] + (i < 32 ? kL11 : J < 2 ? kL21 : kL22) + (i & 31) * kLS + 16 * (J & 1) + 4 * q) =
                            make_float4(x[4 * q], x[4 * q + 1], x[4 * q + 2], x[4 * q + 3]);
                }
            }
            if (query) {
                fence_async_shared();
            } else {
                // the diagonal blocks of 16 of this warp's rows are its own: it inverts them at once
                __syncwarp();
                invert16(s.L[st] + (warp ? kL22 : kL11), lane);
                waits.mark(s);
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&s.lready[st]));
            }
        }
        waits.mark(s);
        warp_arrive(smem_u32(&s.gready[st]), lane);
        named_bar(kBarGate, 128);                 // k.k and q.k have been read
    }
    if (warp == 3) {
        if (elect_lane()) tc_commit(smem_u32(&s.last_kk));
        drain(s.last_kk, 0, p);
    }
    waits.mark(s);
}

// ---------------------------------------------------------------------------
// inverse warps
// ---------------------------------------------------------------------------

// M by blocks of 32 (two of them, half the warps each: steps 0 and 1) and 64 (steps 2, 3 and 4, 5): M21 = -M22 (L21 M11).
// Every step makes four columns of a row of Z = X Y to a thread, from the l in [l0, l1) that a triangle leaves; a warp
// takes a short and a long strip of M11's columns, then of M22's rows.  X, Y, Z: places from s.L on.
constexpr int kInvSteps = 6, kInvWarps = 4;
struct InverseStep {
    int X, Y, Z, l0, l1;
};
__host__ __device__ __forceinline__ InverseStep inverse_step(int step, int L, int warp, int lane)
{
    const int B = L + (warp >> 1 ? kL22 : kL11), T = 2 * kLFloats, T16 = T + (warp >> 1) * 16 * kLS;
    const int strip = 4 * (step & 1 ? 7 - warp : warp);
    if (step < 2) {
        const int in_half = (warp & 1) * 32 + lane, row = in_half >> 2, col = 4 * (in_half & 3), below = B + (16 + row) * kLS;
        return {below + (step ? 16 : 0), (step ? T16 : B) + col, (step ? below : T16 + row * kLS) + col, 0, 16};
    }
    if (step < 4) return {L + kL21 + lane * kLS, L + kL11 + strip, T + lane * kLS + strip, strip, 32};
    const int row = strip + (lane >> 3), col = 4 * (lane & 7);
    return {L + kL22 + row * kLS, T + col, L + kL21 + row * kLS + col, 0, strip + 4};
}
// whether the warps meet behind a step (the last: the next chunk's first products go where the slowest warp still reads these)
__host__ __device__ __forceinline__ bool inverse_joins(int step) { return step < 2 || step == 3 || step == kInvSteps - 1; }

__device__ __forceinline__ void inverse_warps(const PrefillParams &p, PrefillShared &s)
{
    const int tid = threadIdx.x - kInv0, lane = tid & 31, warp = tid >> 5;
    Waits waits{p.polls + 16u * s.total};
#pragma unroll 1
    for (int g = 0; g < s.total; ++g) {
        const int st = g & 1;
        waits.on(s.lready[st], (g >> 1) & 1);
        float *F = &s.L[0][0];
#pragma unroll 1
        for (int step = 0; step < kInvSteps; ++step) {
            const InverseStep at = inverse_step(step, st * kLFloats, warp, lane);
            float acc[4] = {};
#pragma unroll 2
            for (int l = at.l0; l < at.l1; l += 4) {
                const float4 x = *reinterpret_cast<const float4 *>(F + at.X + l);
                const float xe[4] = {x.x, x.y, x.z, x.w};
                float4 y[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) y[e] = *reinterpret_cast<const float4 *>(F + at.Y + (l + e) * kLS);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    acc[0] = fmaf(xe[e], y[e].x, acc[0]);
                    acc[1] = fmaf(xe[e], y[e].y, acc[1]);
                    acc[2] = fmaf(xe[e], y[e].z, acc[2]);
                    acc[3] = fmaf(xe[e], y[e].w, acc[3]);
                }
            }
            const float f = step == 1 || step >= 4 ? -1.f : 1.f;
            *reinterpret_cast<float4 *>(F + at.Z) = make_float4(f * acc[0], f * acc[1], f * acc[2], f * acc[3]);
            if (step == kInvSteps - 1) {
                waits.mark(s);
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&s.inverted[st]));
            }
            if (inverse_joins(step)) named_bar(kBarInv, 32 * kInvWarps);
        }
    }
    waits.mark(s);
}

// ---------------------------------------------------------------------------
// the issuing warps
// ---------------------------------------------------------------------------

// The loops stay rolled: a product's few instructions are fetched once and run from the instruction
// buffer, where straight-line code waits longer for its next line than for the tensor cores.
__device__ __forceinline__ void issue_thread(const PrefillParams &p, PrefillShared &s)
{
    Waits waits{p.polls + 16u * s.total};
    const int total = s.total;
    const bool silent = s.silent;
    bool ok = true;
    auto wait = [&](unsigned long long &bar, uint32_t parity) {
        ok = ok && waits.on(bar, parity);
        tc_fence_after();
        return ok;
    };
    // (Each product adds to its sum with a rounding of some 2^-24 of that sum, towards zero: so the small pieces come first,
    // and few products meet a sum of full size.)
    // U or U A: two FP32 operands of three BF16 pieces each, one pair of which this adds; pair q of six is low times high, high times
    // low, middle times middle, middle times high, high times middle, high times high.  The
    // columns of tokens 0 .. 31 are sums over those tokens alone, and an accumulator of their own: products of one shape on one
    // accumulator keep their order.
    auto pair = [&](uint32_t d, uint32_t a, uint32_t b, int pa, int pb, uint32_t add) {
        constexpr uint32_t lower = 32 * 64 / 16, right = kTriRight / 16, idesc = idesc_bf16_f32(128, kC / 2);
        b += pb * (kTriBytes / 16);
        const uint32_t a0 = a + token_piece(pa, 0), a1 = a + token_piece(pa, 1);
        tc_mma_ts(d, a0, desc_tri(b), idesc, add);
        tc_mma_ts(d, a0 + 8, desc_tri(b + 2), idesc, 1);
        tc_mma_ts(d + kC / 2, a0, desc_tri(b + lower), idesc, add);
        tc_mma_ts(d + kC / 2, a0 + 8, desc_tri(b + lower + 2), idesc, 1);
        tc_mma_ts(d + kC / 2, a1, desc_tri(b + right), idesc, 1);
        tc_mma_ts(d + kC / 2, a1 + 8, desc_tri(b + right + 2), idesc, 1);
    };
    constexpr int kPairA[6] = {2, 0, 1, 1, 0, 0}, kPairB[6] = {0, 2, 1, 0, 1, 0};
    // a piece (0 high, 2 low) of a half of both threads' features of S times the keys (rows 0..63 of the tile) or the queries
    // (64..127)
    auto product = [&](uint32_t d, uint32_t tile, int half, int piece, bool first) {
        const uint32_t b = desc_low(tile) + half * 4, a = kColS + 64 * piece + 16 * half;
        tc_mma_ts(d, a, desc_k(b), idesc_bf16_f32(128, kC), first ? 0u : 1u);
        tc_mma_ts(d, a + 8, desc_k(b + 2), idesc_bf16_f32(128, kC), 1);
        tc_mma_ts(d, a + 32, desc_k(b + 128 * 128 / 16), idesc_bf16_f32(128, kC), 1);
        tc_mma_ts(d, a + 40, desc_k(b + 128 * 128 / 16 + 2), idesc_bf16_f32(128, kC), 1);
    };
#pragma unroll 1
    for (int g = 0; g < total; ++g) {
        const int st = g & 1, sk = g % kStages;
        const uint32_t par = g & 1, par2 = (g >> 1) & 1;
        const uint32_t kq = smem_u32(s.KQ[sk]);
        if (!wait(s.full[sk], (g / kStages) & 1) || !wait(s.gready[st], par2)) break;
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
            if (!wait(s.have_s[half], par)) break;
#pragma unroll 1
            for (int piece = 2; piece >= 0; --piece) product(kColDK, kq, half, piece, half == 0 && piece == 2);
            if (half) tc_commit(smem_u32(&s.done_k));
        }
        if (!silent && g > 0 && !wait(s.read_o, par ^ 1u)) break;
#pragma unroll 1
        for (int q = silent ? 6 : 0; q < 6; ++q) product(kColDQ, kq + kC * 128, q & 1, 2 - (q >> 1), q == 0);
        if (!wait(s.mready[st], par2) || !wait(s.have_x, par)) break;
        {
            const uint32_t b = desc_low(smem_u32(s.M[0]));
            // (Straight-line: the state waits for it, and a rolled loop issues a product in 20 cycles, this in 16, as long as it takes.
            // One prompt of 32768 tokens, 32 heads: 1344 us rolled, 1263 with U A straight-line as well, 1258 so.)
#pragma unroll
            for (int q = 0; q < 6; ++q) pair(kColU, kColX, b, kPairA[q], kPairB[q], (uint32_t)q);
        }
        tc_commit(smem_u32(&s.done_u));
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
            if (!wait(s.have_us[half], par)) break;
            {
                const uint32_t b = desc_low(kq) + half * (16 * 128 / 16);
#pragma unroll
                for (int piece = 2; piece >= 0; --piece) {
                    const uint32_t a = kColS + 32 * piece + 8 * half;
                    tc_mma_ts(kColDK, a, desc_mn(b), idesc_bf16_f32(128, kD) | kBMnMajor, (uint32_t)(half | (piece < 2)));
                    tc_mma_ts(kColDK, a + 16, desc_mn(b + 32 * 128 / 16), idesc_bf16_f32(128, kD) | kBMnMajor, 1);
                }
                if (half) {
                    tc_commit(smem_u32(&s.done_s));
                    tc_commit(smem_u32(&s.empty[sk]));
                }
            }
        }
        if (!silent) {
            if (!wait(s.have_u, par)) break;
            const uint32_t b = desc_low(smem_u32(s.A[st][0]));
#pragma unroll 1
            for (int q = 0; q < 6; ++q) pair(kColU, kColUA, b, (0x052 >> (2 * q)) & 3, (0x118 >> (2 * q)) & 3, (uint32_t)q);   // (kPairA, kPairB)
        }
        tc_commit(smem_u32(&s.done_o));
        tc_commit(smem_u32(&s.gused[st]));
    }
    tc_commit(smem_u32(&s.last));
    drain(s.last, 0, p);   // no product in flight when tensor memory is given back
    waits.mark(s);
}

// M's pieces, eight columns to a thread and turn, two turns to a block of 32 x 32
__device__ __forceinline__ void piece_warps(const PrefillParams &p, PrefillShared &s)
{
    const int tid = threadIdx.x - kIssue0 - 64, lane = tid & 31;
    Waits waits{p.polls + 16u * s.total};
#pragma unroll 1
    for (int g = 0; g < s.total; ++g) {
        const int st = g & 1;
        waits.on(s.inverted[st], (g >> 1) & 1);
        if (g > 0) waits.on(s.done_u, (g & 1) ^ 1u);          // the M before it has been read
#pragma unroll 1
        for (int q = 0; q < 6; ++q) {
            const int row = 16 * (q & 1) + (tid >> 2), col = 8 * (tid & 3);   // in the block
            float x[8];
            read_n(s.L[st] + (q < 2 ? kL11 : q < 4 ? kL21 : kL22) + row * kLS + col, x);
            pieces3<4>(x, [&](int piece, const uint32_t (&w)[4]) {
                *reinterpret_cast<uint4 *>(s.M[piece] + tri_at(row + (q < 2 ? 0 : 32), col + (q < 4 ? 0 : 32))) = make_uint4(w[0], w[1], w[2], w[3]);
            });
        }
        fence_async_shared();
        waits.mark(s);
        __syncwarp();
        if (lane == 0) {
            mbar_arrive(smem_u32(&s.mready[st]));
            mbar_arrive(smem_u32(&s.lfree[st]));
        }
    }
    waits.mark(s);
}

__device__ __forceinline__ void copy_thread(const PrefillParams &p, PrefillShared &s, const CUtensorMap &qmap, const CUtensorMap &kmap,
                                            const CUtensorMap &vmap)
{
    Waits waits{p.polls + 16u * s.total};
    const bool withheld = (p.debug_flags & 1) && blockIdx.x == 0 && p.split.mode != kPieces;
    int g = 0, kq_issued = 0, v_issued = 0;
    bool go = true;
#pragma unroll 1
    for (uint32_t cycle = 0, at; go && (at = item(cycle)) < p.items; ++cycle) {
        const int rank = at / (p.subs * p.H), left = at - rank * p.subs * p.H, sub = left / p.H, h = left - sub * p.H;
        const int r = s.order[rank], pair = r * p.H + h, hk = h / p.group;
        const int row0 = p.off[r], rows = max(request_rows(p, r), 0);
        const Part part = part_of(p, chunks_of(rows), sub);
        const bool affine = p.split.mode == kAhead && sub > 0, unit = affine && !(sub & 1);
        const size_t whole = (size_t)pair * kD * kD;
        const float *from = affine ? nullptr : p.split.mode == kPieces ? split_state(p.split, pair, part.slot, 0) : p.S0 ? p.S0 + whole : nullptr;
        Start start = unit ? kFromOne : from ? kFromState : kFromZero;
        // the states to be noted: behind every piece of a segment; of the first w pieces; behind the last piece
        float *to = affine ? split_state(p.split, pair, part.slot, unit)
                    : p.split.mode == kAhead && part.j ? split_state(p.split, pair, 0, 0)
                    : p.split.mode == kPieces && part.slot < part.j * p.split.w ? nullptr : p.state + whole;
        int piece = affine ? p.split.w + part.slot : 0, note = affine ? piece_start(p, chunks_of(rows), part.j, piece) : part.end;
        if (from && part.end > part.first)        // the state, for when its turn comes
            asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(from), "r"((uint32_t)(kD * kD * sizeof(float))) : "memory");
#pragma unroll 1
        for (int chunk = part.first; go && chunk < part.end; ++chunk, ++g) {
            const int row = row0 + chunk * kC, n = min(rows - chunk * kC, kC);
            const int sk = g % kStages, sv = g & 1;
            const uint32_t kq_bar = smem_u32(&s.full[sk]), v_bar = smem_u32(&s.vfull[sv]), kq = smem_u32(s.KQ[sk]);
            // (told ahead of the wait for room: the gates are asked for a chunk before their keys)
            s.chunk[g % kChunks] = Chunk{from, chunk + 1 == note ? to : nullptr, row, n, affine ? 0 : n, h, start};
            mbar_arrive(smem_u32(&s.told[g & 3]));
            start = kGoesOn;
            if (affine && chunk + 1 == note) {
                note = piece_start(p, chunks_of(rows), part.j, ++piece);
                to += 2 * kD * kD;
            }
            go = g < kStages || waits.on(s.empty[sk], ((g / kStages) & 1) ^ 1u);
            if (!go) break;
            mbar_expect_tx(kq_bar, kKqBytes);
            go = !withheld;
            if (!go) break;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                tma_load_2d(kq + half * 128 * 128, &kmap, hk * kD + 64 * half, row, kq_bar);
                tma_load_2d(kq + half * 128 * 128 + kC * 128, &qmap, hk * kD + 64 * half, row, kq_bar);
            }
            kq_issued = g + 1;
            go = g < 2 || waits.on(s.vempty[sv], ((g >> 1) & 1) ^ 1u);
            if (!go) break;
            if (unit) {                           // no values: zeros lie there
                mbar_arrive(v_bar);
                continue;
            }
            mbar_expect_tx(v_bar, kVBytes);
            tma_load_2d(smem_u32(s.V[sv]), &vmap, h * kD, row, v_bar);
            v_issued = g + 1;
        }
    }
    // no copy into shared memory in flight at the end
    for (int i = max(kq_issued - kStages, 0); i < kq_issued; ++i) drain(s.full[i % kStages], (i / kStages) & 1, p);
    for (int i = max(v_issued - 2, 0); i < v_issued; ++i) drain(s.vfull[i & 1], (i >> 1) & 1, p);
    waits.mark(s);
}

__device__ __forceinline__ void keep_state(const PrefillParams &p, int pair)
{
    if (p.state == p.S0) return;
    const size_t to = (size_t)pair * kD * kD;
#pragma unroll 1
    for (int e = threadIdx.x; e < kD * kD / 4; e += kThreads)
        reinterpret_cast<float4 *>(p.state + to)[e] =
            p.S0 ? reinterpret_cast<const float4 *>(p.S0 + to)[e] : make_float4(0.f, 0.f, 0.f, 0.f);
}

__global__ void __launch_bounds__(kThreads, 1)
    k_gdn_prefill(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                  const __grid_constant__ CUtensorMap vmap, const PrefillParams p)
{
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    PrefillShared &s = *reinterpret_cast<PrefillShared *>(smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u));
    const int tid = threadIdx.x, warp = tid >> 5;
    // What comes next waits for this launch's end, in the SMs that are left.  kPieces waits later, where the states in front are read
    // (what else it reads is older than the launches before it), and lets nothing in: the next call's first launch would be
    // dealt to fewer, busier SMs (one prompt of 2048 tokens x 32 heads, call after call: 127 us so, 122 without).
    if (p.split.mode != kPieces) {
        pdl_wait();
        pdl_launch_dependents();
    }
    static_assert(w12i::kMaxBudget <= kThreads, "a request to a thread");
    const int mine = tid < p.n_req ? request_rows(p, tid) : 0;   // (on its way while the rest is set up)
    if (tid == 0) {
        for (int i = 0; i < 4; ++i) mbar_init(smem_u32(&s.told[i]), 1);
        for (int st = 0; st < kStages; ++st) {
            mbar_init(smem_u32(&s.full[st]), 1);
            mbar_init(smem_u32(&s.empty[st]), 1);
        }
        for (int st = 0; st < 2; ++st) {
            mbar_init(smem_u32(&s.vfull[st]), 1);
            mbar_init(smem_u32(&s.vempty[st]), 8);
            mbar_init(smem_u32(&s.gready[st]), 4);
            mbar_init(smem_u32(&s.gused[st]), 1);
            mbar_init(smem_u32(&s.lready[st]), 2);
            mbar_init(smem_u32(&s.inverted[st]), 4);
            mbar_init(smem_u32(&s.lfree[st]), 2);
            mbar_init(smem_u32(&s.mready[st]), 2);
        }
        for (unsigned long long *b : {&s.bar_kk, &s.done_k, &s.done_u, &s.done_s, &s.done_o, &s.last, &s.last_kk}) mbar_init(smem_u32(b), 1);
        for (unsigned long long *b : {&s.have_s[0], &s.have_s[1], &s.have_us[0], &s.have_us[1], &s.have_x, &s.have_u, &s.read_o}) mbar_init(smem_u32(b), 8);
        s.abort = 0;
        fence_mbar_init();
        prefetch_tmap(&qmap);
        prefetch_tmap(&kmap);
        prefetch_tmap(&vmap);
    }
    if (warp == 0) tmem_alloc(smem_u32(&s.tmem), 512);
    if (tid >= 32 && tid < 32 + kChunks) s.chunk[tid - 32] = Chunk{};   // (what is read of it where a wait has run out)
    {
        // the requests by their rows, and this CTA's chunks
        int32_t *rows = reinterpret_cast<int32_t *>(s.KQ[0]);
        if (tid < p.n_req) {
            rows[tid] = mine;
            if (mine < 0) atomicCAS(p.status, 0, (int32_t)W12_E_INVAL);
        }
        if (tid == 0) s.total = s.silent = 0;
        __syncthreads();
        if (tid < p.n_req) {
            int rank = 0;
#pragma unroll 1
            for (int j = 0; j < p.n_req; ++j) rank += rows[j] > mine || (rows[j] == mine && j < tid);
            s.order[rank] = (uint16_t)tid;
        }
        __syncthreads();
        int chunks = 0;
#pragma unroll 1
        for (uint32_t cycle = tid, at; (at = item(cycle)) < p.items; cycle += kThreads) {
            const int rank = at / (p.subs * p.H);
            const Part part = part_of(p, chunks_of(rows[s.order[rank]]), (at - rank * p.subs * p.H) / p.H);
            chunks += part.end - part.first;
        }
        if (chunks) atomicAdd(&s.total, chunks);
        if (p.split.mode == kWhole) {
            // where there is no token the state stays what it was (those pairs come last)
#pragma unroll 1
            for (uint32_t cycle = 0, at; (at = item(cycle)) < p.items; ++cycle) {
                const int rank = at / (uint32_t)p.H, r = s.order[rank];
                if (rows[r] == 0) keep_state(p, r * p.H + (at - rank * p.H));
            }
        } else if (blockIdx.x < p.items) {        // one item: see above
            const uint32_t at = blockIdx.x;
            const int rank = at / (p.subs * p.H), left = at - rank * p.subs * p.H, sub = left / p.H, h = left - sub * p.H;
            const int r = s.order[rank];
            if (p.split.mode == kAhead) {
                if (sub == 0 && rows[r] == 0) keep_state(p, r * p.H + h);
                if (tid == 0 && sub) s.silent = 1;
                if (sub && !(sub & 1)) {          // P has no values
#pragma unroll 1
                    for (int e = tid; e < (int)(sizeof(s.V) / 16); e += kThreads) reinterpret_cast<uint4 *>(s.V)[e] = make_uint4(0, 0, 0, 0);
                }
            }
        }
    }
    fence_async_shared();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (tid < kToken0) {
        regs_inc<kRegsState>();
        state_warps(p, s);
    } else if (tid < kGate0) {
        token_warps(p, s);
    } else if (tid < kInv0) {
        regs_dec<kRegsGate>();
        gate_warps(p, s);
    } else if (tid < kIssue0) {
        regs_dec<kRegsInv>();
        inverse_warps(p, s);
    } else {
        regs_dec<kRegsIssue>();
        if (warp == kIssue0 / 32 && elect_lane()) issue_thread(p, s);
        if (tid >= kIssue0 + 64) piece_warps(p, s);
        if (tid == kIssue0 + 32) copy_thread(p, s, qmap, kmap, vmap);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (tid == 0 && s.abort) atomicCAS(p.status, 0, (int32_t)W12_E_TIMEOUT);
    if (tid == 0 && p.split.mode == kAhead) {
        const uint32_t a_rank = p.subs * p.H, left = blockIdx.x % a_rank;
        p.split.failed[(s.order[blockIdx.x / a_rank] * p.H + left % p.H) * p.subs + left / p.H] = s.abort;
    }
    if (warp == 0) tmem_dealloc(s.tmem, 512);
}

// The states in front of the pieces, segment after segment: S P + Q over Q.  A CTA takes 8 rows of a pair's states for each of its
// groups of 8 warps (rows are each other's business in no product), so P, which the copy engine brings a product ahead, is
// read once for all of them.  A warp takes 16 of a product's 128 features; its sums join those of the group's other warps
// in shared memory.  8 rows' 131,072 multiplications take 0.55 us of an SM, as long as P's way from L2.
constexpr int kJoinRows = 8, kJoinWarps = 8;      // of a group
template <int kGroups>
struct JoinShared {
    float P[2][kD][kD];
    float S[kGroups][kD][kJoinRows + 4];          // the state in front, by features, 12 banks apart
    float sums[kGroups][kJoinWarps][kJoinRows][kD];
    unsigned long long full[2];
};

// a plain copy into shared memory, addresses and size multiples of 16 bytes
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src), "r"(bytes),
                 "r"(bar)
                 : "memory");
}

template <int kGroups>
__global__ void __launch_bounds__(32 * kJoinWarps * kGroups, 1) k_gdn_join(const PrefillParams p)
{
    pdl_wait();                                   // first of all: the launch behind this one counts on it
    pdl_launch_dependents();
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    JoinShared<kGroups> &s = *reinterpret_cast<JoinShared<kGroups> *>(smem_raw);
    constexpr int kOwn = kD / kJoinWarps;         // features of a warp
    const int tid = threadIdx.x & 255, lane = tid & 31, warp = tid >> 5, group = threadIdx.x >> 8;
    const int pair = blockIdx.y, row0 = (blockIdx.x * kGroups + group) * kJoinRows, w = p.split.w;
    const int last = split_segments(chunks_of(request_rows(p, pair / p.H)), p.split.j, w) * w;
    if (last == 0) return;
    if (threadIdx.x == 0) {
        mbar_init(smem_u32(&s.full[0]), 1);
        mbar_init(smem_u32(&s.full[1]), 1);
        fence_mbar_init();
    }
    auto fetch = [&](int slot) {                  // thread 0
        const uint32_t bar = smem_u32(&s.full[slot & 1]);
        fence_async_shared();                     // (behind what has been read there)
        mbar_expect_tx(bar, kD * kD * 4);
        bulk_load(smem_u32(s.P[slot & 1]), split_state(p.split, pair, slot, 1), kD * kD * 4, bar);
    };
    const int row = 4 * (tid >> 7), col = tid & 127;   // of this thread's four sums
    float *Q = split_state(p.split, pair, 0, 0) + (row0 + row) * kD + col;
    auto read_q = [&]() { return make_float4(Q[0], Q[kD], Q[2 * kD], Q[3 * kD]); };
    float(&S)[kD][kJoinRows + 4] = s.S[group];
    *reinterpret_cast<float4 *>(&S[col][row]) = read_q();
    if (threadIdx.x == 0) fetch(1);
    __syncthreads();
    Waits waits{p.polls};
#pragma unroll 1
    for (int slot = 1, piece = 1; slot <= last; ++slot, ++piece) {
        if (threadIdx.x == 0 && slot < last) fetch(slot + 1);
        Q += 2 * kD * kD;                         // (a piece's states lie behind those of the one before)
        float4 sum = read_q();
        float2 acc[kJoinRows / 2][4] = {};        // of two rows (which lie beside one another: four values doubled a feature, not eight)
        waits.on(s.full[slot & 1], ((slot - 1) >> 1) & 1);
#pragma unroll
        for (int l = 0; l < kOwn; ++l) {
            float x[kJoinRows];
            read_n(S[warp * kOwn + l], x);
            const float4 y = *reinterpret_cast<const float4 *>(&s.P[slot & 1][warp * kOwn + l][4 * lane]);
#pragma unroll
            for (int r = 0; r < kJoinRows / 2; ++r) {
                const float2 rows = make_float2(x[2 * r], x[2 * r + 1]);
                acc[r][0] = __ffma2_rn(rows, make_float2(y.x, y.x), acc[r][0]);
                acc[r][1] = __ffma2_rn(rows, make_float2(y.y, y.y), acc[r][1]);
                acc[r][2] = __ffma2_rn(rows, make_float2(y.z, y.z), acc[r][2]);
                acc[r][3] = __ffma2_rn(rows, make_float2(y.w, y.w), acc[r][3]);
            }
        }
#pragma unroll
        for (int r = 0; r < kJoinRows / 2; ++r) {
            float(*sums)[kD] = &s.sums[group][warp][2 * r];
            *reinterpret_cast<float4 *>(&sums[0][4 * lane]) = make_float4(acc[r][0].x, acc[r][1].x, acc[r][2].x, acc[r][3].x);
            *reinterpret_cast<float4 *>(&sums[1][4 * lane]) = make_float4(acc[r][0].y, acc[r][1].y, acc[r][2].y, acc[r][3].y);
        }
        __syncthreads();
#pragma unroll
        for (int v = 0; v < kJoinWarps; ++v) {
            sum.x += s.sums[group][v][row][col];
            sum.y += s.sums[group][v][row + 1][col];
            sum.z += s.sums[group][v][row + 2][col];
            sum.w += s.sums[group][v][row + 3][col];
        }
        Q[0] = sum.x;
        Q[kD] = sum.y;
        Q[2 * kD] = sum.z;
        Q[3 * kD] = sum.w;
        if (piece == w) {                         // the state in front of the next segment
            *reinterpret_cast<float4 *>(&S[col][row]) = sum;
            piece = 0;
        }
        __syncthreads();
    }
    if (waits.left == 0) {                        // (a copy did not come: no piece of the pair is run)
        atomicCAS(p.status, 0, (int32_t)W12_E_TIMEOUT);
        p.split.failed[pair * (2 * p.split.j + 1)] = 1;
        if (threadIdx.x == 0) {
            drain(s.full[0], ((last >> 1) + 1) & 1, p);
            drain(s.full[1], (((last + 1) >> 1) + 1) & 1, p);
        }
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
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(f);
    }
    return fn;
}

// Segments and their pieces for so many pairs of a call's rows: what the SMs take of both launches' items.
constexpr size_t kSplitHeader = 4096;             // a word for each item of kAhead
void split_of(int num_sms, int64_t pairs, int32_t n_rows, int32_t &j, int32_t &w)
{
    const int most = (int)std::min<int64_t>(std::min<int64_t>(num_sms, kSplitHeader / sizeof(int32_t)) / pairs, 64);   // CTAs a pair
    j = (most - 1) / 2;
    w = j > 0 ? std::min((most - 1) / j, 3) : 0;
    if (j > 0) j = split_segments((int)(((int64_t)n_rows + kC - 1) / kC), j, w);
}

}  // namespace

namespace w12i {

int launch_gdn_prefill(const GdnSeqArgs &a, void *stream)
{
    CUtensorMap maps[3] = {};
    if (a.n_rows > 0) {
        EncodeTiledFn enc = encode_fn();
        if (!enc) return (int)cudaErrorNotSupported;
        const uint16_t *src[3] = {a.q, a.k, a.v};
        const int64_t stride[3] = {a.q_stride, a.k_stride, a.v_stride};
        for (int i = 0; i < 3; ++i) {
            const cuuint64_t dims[2] = {(cuuint64_t)(i < 2 ? a.Hk : a.H) * kD, (cuuint64_t)a.n_rows};
            const cuuint64_t strides[1] = {(cuuint64_t)stride[i] * 2};
            const cuuint32_t box[2] = {i < 2 ? 64u : (cuuint32_t)kD, (cuuint32_t)kC}, estr[2] = {1, 1};
            if (enc(&maps[i], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<uint16_t *>(src[i]), dims, strides, box, estr,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, i < 2 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
                return (int)cudaErrorInvalidValue;
        }
    }
    static std::atomic<int> known{0};
    int regs = known.load(std::memory_order_relaxed);
    if (regs == 0) {
        cudaFuncAttributes attr{};
        const cudaError_t e = cudaFuncGetAttributes(&attr, k_gdn_prefill);
        if (e != cudaSuccess) return (int)e;
        known.store(regs = attr.numRegs, std::memory_order_relaxed);
    }
    if (regs < kRegsLaunch) return (int)cudaErrorInvalidConfiguration;   // the register shares need that many
    PrefillParams p{};
    p.S0 = a.S0;
    p.state = a.state;
    p.o = a.o;
    p.alpha = a.alpha;
    p.beta = a.beta;
    p.off = a.off;
    p.H = a.H;
    p.group = a.H / a.Hk;
    p.n_req = a.n_req;
    p.n_rows = a.n_rows;
    p.polls = (uint32_t)std::min<uint64_t>(a.timeout_ns / kWaitSleepNs + 1, 1u << 30);
    p.status = a.status;
    p.debug_flags = a.debug_flags;
    cudaLaunchConfig_t cfg{};
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = sizeof(PrefillShared) + 1024;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaFuncSetAttribute(k_gdn_prefill, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)cfg.dynamicSmemBytes);
    if (e != cudaSuccess) return (int)e;
    const int64_t pairs = (int64_t)a.n_req * a.H;
    cudaLaunchAttribute behind{};                 // each launch begins while the one before it ends, and waits for that
    behind.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    behind.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &behind;
    cfg.numAttrs = 1;
    auto run = [&](Mode mode, int subs) {
        p.split.mode = mode;
        p.subs = (uint32_t)subs;
        p.items = (uint32_t)(pairs * subs);
        cfg.gridDim = dim3((uint32_t)std::min<int64_t>(p.items, a.num_sms));   // one CTA fills an SM
        return cudaLaunchKernelEx(&cfg, k_gdn_prefill, maps[0], maps[1], maps[2], p);
    };
    if (a.scratch) split_of(a.num_sms, pairs, a.n_rows, p.split.j, p.split.w);
    if (p.split.j == 0) return (int)run(kWhole, 1);
    p.split.failed = static_cast<int32_t *>(a.scratch);
    p.split.states = reinterpret_cast<float *>(static_cast<uint8_t *>(a.scratch) + kSplitHeader);
    if ((e = run(kAhead, 2 * p.split.j + 1)) != cudaSuccess) return (int)e;
    // Two groups halve P's ways from L2, which bound it where there are many rows; one is the faster where SMs are left.  (Four
    // requests of up to 4096 tokens, 4 heads: 115 us a call with one group, 114 with two; one such request: 82 and 95.)
    auto join = [&](auto kernel, int groups, size_t bytes) {
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
        if (e != cudaSuccess) return e;
        cudaLaunchConfig_t c{};
        c.gridDim = dim3(kD / kJoinRows / groups, (uint32_t)pairs);
        c.blockDim = dim3(32 * kJoinWarps * groups);
        c.dynamicSmemBytes = bytes;
        c.stream = cfg.stream;
        c.attrs = &behind;
        c.numAttrs = 1;
        return cudaLaunchKernelEx(&c, kernel, p);
    };
    e = pairs * (kD / kJoinRows) > a.num_sms ? join(k_gdn_join<2>, 2, sizeof(JoinShared<2>)) : join(k_gdn_join<1>, 1, sizeof(JoinShared<1>));
    if (e != cudaSuccess) return (int)e;
    return (int)run(kPieces, p.split.j * p.split.w + 1);
}

size_t gdn_scratch_bytes(int num_sms, int32_t H, int32_t n_rows)
{
    int j = 0, w;
    for (int64_t pairs = H; j == 0 && pairs <= num_sms; pairs += H) split_of(num_sms, pairs, n_rows, j, w);
    return j ? kSplitHeader + (size_t)num_sms * 2 * kD * kD * sizeof(float) : 0;
}

// Words that two of the inverse's warps touch, one of them writing, with no meeting in between: two chunks' steps on end, as the
// warps take them.  (What is not theirs waits for barriers of its own.)
int gdn_inverse_conflicts()
{
    constexpr int kWords = 2 * kLFloats + 32 * kLS;
    std::vector<uint8_t> read(kWords), written(kWords);        // a bit for each warp, since the last meeting
    int conflicts = 0;
    for (int chunk = 0; chunk < 2; ++chunk)
        for (int step = 0; step < kInvSteps; ++step) {
            for (int warp = 0; warp < kInvWarps; ++warp)
                for (int lane = 0; lane < 32; ++lane) {
                    const InverseStep at = inverse_step(step, chunk * kLFloats, warp, lane);
                    const uint8_t own = (uint8_t)(1 << warp);
                    for (int e = 0; e < 4; ++e) {
                        for (int l = at.l0; l < at.l1; ++l) read[at.Y + l * kLS + e] |= own;
                        written[at.Z + e] |= own;
                    }
                    for (int l = at.l0; l < at.l1; ++l) read[at.X + l] |= own;
                }
            if (!inverse_joins(step) && !(chunk && step == kInvSteps - 1)) continue;
            for (int w = 0; w < kWords; ++w) {
                const int writers = written[w], all = writers | read[w];
                conflicts += writers && (all & (all - 1));
                written[w] = read[w] = 0;
            }
        }
    return conflicts;
}

}  // namespace w12i
