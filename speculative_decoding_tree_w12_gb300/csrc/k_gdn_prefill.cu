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
// One CTA to a (request, head); the state rows c lie on the 128 lanes of tensor
// memory throughout, so that all its products take their left operand from
// there and no operand but M and A is ever written to shared memory:
//     D_K[c][j] = S k_j    D_Q[c][j] = S q_j    U[c][i] = X M^T    U A^T    S' += U K.
// A product's FP32 side (S, X, U, M, A) is taken as three BF16 pieces that add up to
// it exactly, keys and queries as they are, all with FP32 accumulation: two
// pieces (2^-17) would be the largest error of the layer by far.  Products of
// two FP32 sides take the six pairs of pieces above 2^-24.
//
// Sixteen warps:
//  * state warps (0..7; two threads to a state row, each with half of the
//    columns; S itself stays in their registers) turn accumulators into operands,
//  * chunk warps (8..11) make M and A of the next chunk: k.k and q.k on the
//    tensor cores, then the inverse of two 32 x 32 blocks by columns and of the
//    block below them from those two,
//  * warp 12 issues the state warps' products, warp 13 the copies by TMA.
// Every wait is bounded: a wait that runs out sets s.abort, which ends every
// other wait at once, so all roles run to their ends; the state is then left
// unwritten.
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>

#include "w12_device.cuh"

using namespace w12d;

namespace {

constexpr int kD = 128;             // head dimension
constexpr int kC = 64;              // tokens of a chunk
constexpr int kThreads = 512;
constexpr int kStateWarps = 8;
constexpr int kChunkThreads = 128;
constexpr int kRegsLaunch = 128, kRegsState = 176, kRegsChunk = 104, kRegsIssue = 40;
static_assert(256 * kRegsState + 128 * kRegsChunk + 128 * kRegsIssue <= kThreads * kRegsLaunch, "register shares");

// tensor memory columns
constexpr uint32_t kColS = 0;       // S: three pieces of 64 columns; later U's pieces, first scaled for S', then for A
constexpr uint32_t kColDQ = 192;    // S q
constexpr uint32_t kColDK = 256;    // S k; then X's low piece; then, with the next 64 columns, U K
constexpr uint32_t kColX = 320;     // X's high and middle pieces
constexpr uint32_t kColU = 384;     // U; then U A
constexpr uint32_t kColKK = 448;    // k.k (lanes 0..63) and q.k (lanes 64..127) of the next chunk

constexpr int kLS = 68;             // FP32 row stride of L and M (16-byte rows, 4 banks apart)
constexpr int kTS = 36;
constexpr int kBarChunk = 1;        // named barrier of the chunk warps

struct PrefillShared {
    uint8_t KQ[2][2 * 128 * 128];   // [stage][feature half][key rows, query rows][64 BF16], 128-byte swizzle
    uint8_t M[2][3][kC * 128];      // pieces of M and A, rows of 64 BF16, 128-byte swizzle
    uint8_t A[2][3][kC * 128];
    uint16_t V[2][kC * kD];
    float L[kC * kLS];
    float T[32 * kTS];
    float a[kC];
    float b[4][kC], G[4][kC], tail[4][kC];   // of chunk c in [c % 4]: strengths, G_i, D_Ci
    unsigned long long full[2], empty[2], ready[2];
    unsigned long long bar_kk;
    unsigned long long have_s, have_x, have_us, have_u, read_o;   // to the issuing warp: operands written, outputs read
    unsigned long long done_k, done_u, done_s, done_o;            // from it: products done
    unsigned long long last, last_kk;
    uint32_t tmem;
    int32_t abort;
};
static_assert(sizeof(PrefillShared) + 1024 <= 227 * 1024, "shared memory above the per-CTA limit");
constexpr uint32_t kStageBytes = sizeof(PrefillShared::KQ) / 2 + sizeof(PrefillShared::V) / 2;

struct PrefillParams {
    const float *S0;                // may be null: zero
    float *state, *o;
    const float *alpha, *beta;
    const int32_t *off;
    int32_t H, group, n_rows;
    uint64_t timeout_ns;
    int32_t *status;
    int32_t debug_flags;            // bit 0: CTA (0, 0) announces its first copies and leaves them out (test hook)
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

__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

// D[tmem] (+)= A[smem] * B[smem], one elected lane of a converged warp (a product issued from a
// diverged thread takes 124 cycles to issue on GB300, an elected one none beyond its own time)
__device__ __forceinline__ void tc_mma_ss_elect(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                                uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred e, p;\n\telect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// BF16 operand whose rows (of 64 features, 128-byte swizzle) are its K index: 8-row groups 1024 bytes
// apart, the next 64 features `half` bytes on
__device__ __forceinline__ uint64_t smem_desc_mn_sw128(uint32_t saddr, uint32_t half)
{
    uint64_t d = 0;
    d |= (uint64_t)((saddr >> 4) & 0x3FFFu);
    d |= (uint64_t)(half >> 4) << 16;
    d |= (uint64_t)(1024u >> 4) << 32;
    d |= (uint64_t)1u << 46;
    d |= (uint64_t)2u << 61;
    return d;
}

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
            const uint32_t b0 = __float_as_uint(x[2 * i]), b1 = __float_as_uint(x[2 * i + 1]);
            w[i] = __byte_perm(b0, b1, 0x7632);
            if (piece < 2) {
                const float2 r = __ffma2_rn(make_float2(__uint_as_float(b0 & 0xffff0000u), __uint_as_float(b1 & 0xffff0000u)),
                                            make_float2(-1.f, -1.f), make_float2(x[2 * i], x[2 * i + 1]));
                x[2 * i] = r.x;
                x[2 * i + 1] = r.y;
            }
        }
        put(piece, w);
    }
}

// 32 lanes x 32 columns as floats, the load complete
__device__ __forceinline__ void tmem_read(uint32_t taddr, float (&x)[32])
{
    uint32_t w[32];
    tmem_ld_x32(taddr, w);
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 32; ++i) x[i] = __uint_as_float(w[i]);
}

// this warp's tensor-memory accesses are done: one arrival for the warp
__device__ __forceinline__ void warp_arrive(uint32_t bar, int lane)
{
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
}

// a wait that nothing ends early: for what is in flight at the end
__device__ __forceinline__ void drain(uint32_t bar, uint32_t parity, uint64_t timeout_ns)
{
    const uint64_t t0 = globaltimer();
    while (!mbar_try_wait(bar, parity) && globaltimer() - t0 < timeout_ns) {
    }
}

struct Tile {
    int32_t row0, n, chunks;        // the request's first row, its rows, chunks
};

// ---------------------------------------------------------------------------
// state warps
// ---------------------------------------------------------------------------

__device__ __forceinline__ void put_state(float (&S)[64], uint32_t tm, int hs)
{
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        float x[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) x[i] = S[32 * q + i];
        pieces3<16>(x, [&](int piece, const uint32_t (&w)[16]) { tmem_st_x16(tm + kColS + 64 * piece + 32 * hs + 16 * q, w); });
    }
    tmem_st_wait();
}

__device__ __forceinline__ void state_warps(const PrefillParams &p, PrefillShared &s, const Tile &t, int r, int h)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, hs = warp >> 2;
    const int c = (warp & 3) * 32 + lane;                                 // state row
    const uint32_t tm = s.tmem + ((uint32_t)((warp & 3) * 32) << 16);     // this warp's lanes
    auto wait = [&](unsigned long long &bar, uint32_t parity) {
        mbar_wait(smem_u32(&bar), parity, p.timeout_ns, p.status, &s.abort);
        tc_fence_after();
    };
    const size_t at = (((size_t)r * p.H + h) * kD + c) * kD + 64 * hs;    // this thread's half row
    float S[64];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const float4 x = p.S0 ? *reinterpret_cast<const float4 *>(p.S0 + at + 4 * i) : make_float4(0.f, 0.f, 0.f, 0.f);
        S[4 * i] = x.x;
        S[4 * i + 1] = x.y;
        S[4 * i + 2] = x.z;
        S[4 * i + 3] = x.w;
    }
    put_state(S, tm, hs);
    warp_arrive(smem_u32(&s.have_s), lane);
#pragma unroll 1
    for (int ch = 0; ch < t.chunks; ++ch) {
        const int st = ch & 1, k4 = ch & 3;
        const uint32_t par = ch & 1, par2 = (ch >> 1) & 1;
        float x[32];
        // X = b (v - G S k): tokens 32 hs .. 32 hs + 31
        wait(s.full[st], par2);
        wait(s.ready[st], par2);
        wait(s.done_k, par);
        tmem_read(tm + kColDK + 32 * hs, x);
        {
            const uint16_t *v = s.V[st] + 32 * hs * kD + c;
            const float *b = s.b[k4] + 32 * hs, *G = s.G[k4] + 32 * hs;
#pragma unroll
            for (int j = 0; j < 32; ++j)
                x[j] = b[j] * (__uint_as_float((uint32_t)v[j * kD] << 16) - G[j] * x[j]);
        }
        // (the low piece goes where this thread has read S k: the other half's columns may not be read yet)
        pieces3<16>(x, [&](int piece, const uint32_t (&w)[16]) {
            tmem_st_x16(piece < 2 ? tm + kColX + 32 * piece + 16 * hs : tm + kColDK + 32 * hs, w);
        });
        tmem_st_wait();
        warp_arrive(smem_u32(&s.have_x), lane);

        // U, scaled for S' (S's pieces have been read: S q came before U), then for A
        wait(s.done_u, par);
        tmem_read(tm + kColU + 32 * hs, x);
        {
            float y[32];
            const float *tail = s.tail[k4] + 32 * hs;
#pragma unroll
            for (int j = 0; j < 32; ++j) y[j] = x[j] * tail[j];
            pieces3<16>(y, [&](int piece, const uint32_t (&w)[16]) { tmem_st_x16(tm + kColS + 32 * piece + 16 * hs, w); });
        }
        tmem_st_wait();
        warp_arrive(smem_u32(&s.have_us), lane);
        pieces3<16>(x, [&](int piece, const uint32_t (&w)[16]) { tmem_st_x16(tm + kColS + 96 + 32 * piece + 16 * hs, w); });
        tmem_st_wait();
        warp_arrive(smem_u32(&s.have_u), lane);

        // S' = G_C S + U K: features 64 hs .. 64 hs + 63
        const float gc = s.G[k4][kC - 1];
        wait(s.done_s, par);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            tmem_read(tm + kColDK + 64 * hs + 32 * q, x);
#pragma unroll
            for (int i = 0; i < 32; ++i) S[32 * q + i] = fmaf(gc, S[32 * q + i], x[i]);
        }
        wait(s.done_o, par);
        if (ch + 1 < t.chunks) {
            put_state(S, tm, hs);
            warp_arrive(smem_u32(&s.have_s), lane);
        }
        // o = G S q + U A
        float y[32];
        tmem_read(tm + kColDQ + 32 * hs, x);
        tmem_read(tm + kColU + 32 * hs, y);
        warp_arrive(smem_u32(&s.read_o), lane);
        const int left = t.n - ch * kC - 32 * hs;
        float *dst = p.o + ((size_t)(t.row0 + ch * kC + 32 * hs) * p.H + h) * kD + c;
        const size_t step = (size_t)p.H * kD;
        const float *G = s.G[k4] + 32 * hs;
#pragma unroll
        for (int j = 0; j < 32; ++j)
            if (j < left) dst[j * step] = fmaf(G[j], x[j], y[j]);
    }
    if (!*(volatile int32_t *)&s.abort) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            *reinterpret_cast<float4 *>(p.state + at + 4 * i) = make_float4(S[4 * i], S[4 * i + 1], S[4 * i + 2], S[4 * i + 3]);
    }
}

// ---------------------------------------------------------------------------
// chunk warps
// ---------------------------------------------------------------------------

// C (32 x 32) = -/+ X Y of three 32 x 32 blocks in shared memory: two rows and four columns to a thread
template <bool kNeg>
__device__ __forceinline__ void block_product(const float *X, int xs, const float *Y, int ys, float *Z, int zs, int t)
{
    const int r0 = 2 * (t >> 3), c0 = 4 * (t & 7);
    float acc[2][4] = {};
#pragma unroll
    for (int l = 0; l < 32; l += 4) {
        float xr[2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float4 v = *reinterpret_cast<const float4 *>(X + (r0 + i) * xs + l);
            xr[i][0] = v.x;
            xr[i][1] = v.y;
            xr[i][2] = v.z;
            xr[i][3] = v.w;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float4 v = *reinterpret_cast<const float4 *>(Y + (l + e) * ys + c0);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                acc[i][0] = fmaf(xr[i][e], v.x, acc[i][0]);
                acc[i][1] = fmaf(xr[i][e], v.y, acc[i][1]);
                acc[i][2] = fmaf(xr[i][e], v.z, acc[i][2]);
                acc[i][3] = fmaf(xr[i][e], v.w, acc[i][3]);
            }
        }
    }
    const float f = kNeg ? -1.f : 1.f;
#pragma unroll
    for (int i = 0; i < 2; ++i)
        *reinterpret_cast<float4 *>(Z + (r0 + i) * zs + c0) =
            make_float4(f * acc[i][0], f * acc[i][1], f * acc[i][2], f * acc[i][3]);
}

// words of three pieces of 32 values into row `row` of three swizzled tiles, from column `col0` on (a multiple of 32)
__device__ __forceinline__ void put_row(uint8_t (&tile)[3][kC * 128], int row, int col0, float (&x)[32])
{
    pieces3<16>(x, [&](int piece, const uint32_t (&w)[16]) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
            *reinterpret_cast<uint4 *>(tile[piece] + row * 128 + (((col0 / 8 + q) ^ (row & 7)) << 4)) =
                make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
    });
}

__device__ __forceinline__ void chunk_warps(const PrefillParams &p, PrefillShared &s, const Tile &t, int h)
{
    const int tid = threadIdx.x - 256, lane = tid & 31, warp = tid >> 5;
    const int i = tid & 63;                       // token of the chunk
    const bool query = tid >= 64;                 // this thread's row of k.k / q.k
    const uint32_t tm = s.tmem + ((uint32_t)(warp * 32) << 16);
    auto gate = [&](int ch) {                     // threads 0..63: the gate of their token, others its strength; 1 and 0 behind the end
        const int row = ch * kC + i;
        if (row >= t.n) return query ? 0.f : 1.f;
        return (query ? p.beta : p.alpha)[(size_t)(t.row0 + row) * p.H + h];
    };
    float ab = gate(0);
#pragma unroll 1
    for (int ch = 0; ch < t.chunks; ++ch) {
        const int st = ch & 1, k4 = ch & 3;
        const uint32_t par = ch & 1, par2 = (ch >> 1) & 1;
        mbar_wait(smem_u32(&s.full[st]), par2, p.timeout_ns, p.status, &s.abort);
        const int valid = min(t.n - ch * kC, kC);
        if (valid < kC) {
            // rows behind the request's end are another request's, or none: whatever they hold becomes zero
            for (int e = tid; e < (kC - valid) * 16; e += kChunkThreads) {
                const int row = valid + (e >> 4), q = e & 15;
                const uint4 z = make_uint4(0, 0, 0, 0);
                uint8_t *half = s.KQ[st] + (q >> 3) * (128 * 128);
                *reinterpret_cast<uint4 *>(half + row * 128 + (q & 7) * 16) = z;
                *reinterpret_cast<uint4 *>(half + (kC + row) * 128 + (q & 7) * 16) = z;
                *reinterpret_cast<uint4 *>(s.V[st] + row * kD + q * 8) = z;
            }
            fence_async_shared();
        }
        if (query)
            s.b[k4][i] = ab;
        else
            s.a[i] = ab;
        tc_fence_before();
        named_bar(kBarChunk, kChunkThreads);
        if (ch + 1 < t.chunks) ab = gate(ch + 1);
        if (warp == 0) {
            tc_fence_after();
            const uint32_t kq = smem_u32(s.KQ[st]);
            const uint64_t x0 = smem_desc_sw128(kq), x1 = smem_desc_sw128(kq + 128 * 128);
#pragma unroll
            for (int ks = 0; ks < 8; ++ks) {
                const uint64_t d = (ks < 4 ? x0 : x1) + (uint64_t)((ks & 3) * 2);
                tc_mma_ss_elect(s.tmem + kColKK, d, d, idesc_bf16_f32(128, kC), ks ? 1u : 0u);
            }
            tc_commit_elect(smem_u32(&s.bar_kk));
        }
        mbar_wait(smem_u32(&s.bar_kk), par, p.timeout_ns, p.status, &s.abort);
        tc_fence_after();
        const float bi = s.b[k4][i];
        float d = 1.f;                            // D_ij, from j = i down
#pragma unroll
        for (int half = 1; half >= 0; --half) {
            float x[32];
            tmem_read(tm + kColKK + 32 * half, x);
#pragma unroll
            for (int jj = 31; jj >= 0; --jj) {
                const int j = 32 * half + jj;
                if (j + 1 <= kC - 1 && j < i) d *= s.a[j < kC - 1 ? j + 1 : j];
                x[jj] = (query ? j <= i : j < i) ? x[jj] * (query ? d : d * bi) : 0.f;
                if (tid == kC - 1) s.tail[k4][j] = d;
            }
            if (query) {
                put_row(s.A[st], i, 32 * half, x);
            } else {
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    *reinterpret_cast<float4 *>(s.L + i * kLS + 32 * half + 4 * q) =
                        make_float4(x[4 * q], x[4 * q + 1], x[4 * q + 2], x[4 * q + 3]);
            }
        }
        if (!query) s.G[k4][i] = d * s.a[0];
        named_bar(kBarChunk, kChunkThreads);
        // the inverse of the two diagonal blocks, a column to a thread: x_i = [i = j] - sum over l < i of L_il x_l
        if (!query) {
            float *B = s.L + warp * 32 * (kLS + 1);
            float x[32];
#pragma unroll
            for (int row = 0; row < 32; ++row) {
                float acc[4] = {row == lane ? 1.f : 0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int l = 0; l < row; l += 4) {
                    const float4 v = *reinterpret_cast<const float4 *>(B + row * kLS + l);
                    acc[0] = fmaf(-v.x, x[l], acc[0]);
                    if (l + 1 < row) acc[1] = fmaf(-v.y, x[l + 1], acc[1]);
                    if (l + 2 < row) acc[2] = fmaf(-v.z, x[l + 2], acc[2]);
                    if (l + 3 < row) acc[3] = fmaf(-v.w, x[l + 3], acc[3]);
                }
                x[row] = (acc[0] + acc[1]) + (acc[2] + acc[3]);
            }
            __syncwarp();
#pragma unroll
            for (int row = 0; row < 32; ++row) B[row * kLS + lane] = x[row];
        }
        named_bar(kBarChunk, kChunkThreads);
        // and of the block below them: M21 = -M22 (L21 M11)
        block_product<false>(s.L + 32 * kLS, kLS, s.L, kLS, s.T, kTS, tid);
        named_bar(kBarChunk, kChunkThreads);
        block_product<true>(s.L + 32 * (kLS + 1), kLS, s.T, kTS, s.L + 32 * kLS, kLS, tid);
        named_bar(kBarChunk, kChunkThreads);
        {
            const int row = tid >> 1, c0 = (tid & 1) * 32;
            float x[32];
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const float4 v = *reinterpret_cast<const float4 *>(s.L + row * kLS + c0 + 4 * q);
                x[4 * q] = v.x;
                x[4 * q + 1] = v.y;
                x[4 * q + 2] = v.z;
                x[4 * q + 3] = v.w;
            }
            put_row(s.M[st], row, c0, x);
        }
        fence_async_shared();
        warp_arrive(smem_u32(&s.ready[st]), lane);
    }
    if (warp == 0) {
        tc_commit_elect(smem_u32(&s.last_kk));
        drain(smem_u32(&s.last_kk), 0, p.timeout_ns);
    }
}

// ---------------------------------------------------------------------------
// the issuing warps
// ---------------------------------------------------------------------------

// The six pairs of pieces of two FP32 operands, K = 64 tokens: piece columns a[piece] + step, tiles of `B`
template <class F>
__device__ __forceinline__ void issue_pairs(uint32_t d, F a, const uint8_t (*B)[kC * 128])
{
    constexpr int pa[6] = {0, 0, 1, 1, 0, 2}, pb[6] = {0, 1, 0, 1, 2, 0};
#pragma unroll
    for (int q = 0; q < 6; ++q) {
        const uint64_t b = smem_desc_sw128(smem_u32(B[pb[q]]));
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
            tc_mma_ts_elect(d, a(pa[q], ks), b + (uint64_t)(ks * 2), idesc_bf16_f32(128, kC), (q | ks) ? 1u : 0u);
    }
}

__device__ __forceinline__ void issue_warp(const PrefillParams &p, PrefillShared &s, const Tile &t)
{
    const uint32_t tm = s.tmem;
    bool ok = true;
    auto wait = [&](unsigned long long &bar, uint32_t parity) {
        ok = ok && __all_sync(0xffffffffu, mbar_wait(smem_u32(&bar), parity, p.timeout_ns, p.status, &s.abort));
        tc_fence_after();
        return ok;
    };
#pragma unroll 1
    for (int ch = 0; ch < t.chunks; ++ch) {
        const int st = ch & 1;
        const uint32_t par = ch & 1, par2 = (ch >> 1) & 1;
        const uint32_t kq = smem_u32(s.KQ[st]);
        if (!wait(s.full[st], par2) || !wait(s.ready[st], par2) || !wait(s.have_s, par)) break;
        // S k (rows 0..63 of the tile), then S q (rows 64..127) once the last chunk's outputs are read
        auto products = [&](uint32_t d, uint32_t row0) {
            const uint64_t b0 = smem_desc_sw128(kq + row0 * 128), b1 = smem_desc_sw128(kq + 128 * 128 + row0 * 128);
#pragma unroll
            for (int piece = 0; piece < 3; ++piece)
#pragma unroll
                for (int ks = 0; ks < 8; ++ks)
                    tc_mma_ts_elect(d, tm + kColS + 64 * piece + 8 * ks, (ks < 4 ? b0 : b1) + (uint64_t)((ks & 3) * 2),
                                    idesc_bf16_f32(128, kC), (piece | ks) ? 1u : 0u);
        };
        products(tm + kColDK, 0);
        tc_commit_elect(smem_u32(&s.done_k));
        if (ch > 0 && !wait(s.read_o, par ^ 1u)) break;
        products(tm + kColDQ, kC);
        if (!wait(s.have_x, par)) break;
        issue_pairs(tm + kColU, [&](int piece, int ks) {
            return piece < 2 ? tm + kColX + 32 * piece + 8 * ks : tm + kColDK + 8 * (ks & 2) + 8 * ks;
        }, s.M[st]);
        tc_commit_elect(smem_u32(&s.done_u));
        if (!wait(s.have_us, par)) break;
#pragma unroll
        for (int piece = 0; piece < 3; ++piece)
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
                tc_mma_ts_elect(tm + kColDK, tm + kColS + 32 * piece + 8 * ks,
                                smem_desc_mn_sw128(kq + ks * 16 * 128, 128 * 128), idesc_bf16_f32(128, kD) | kBMnMajor,
                                (piece | ks) ? 1u : 0u);
        tc_commit_elect(smem_u32(&s.done_s));
        if (!wait(s.have_u, par)) break;
        issue_pairs(tm + kColU, [&](int piece, int ks) { return tm + kColS + 96 + 32 * piece + 8 * ks; }, s.A[st]);
        tc_commit_elect(smem_u32(&s.done_o));
        tc_commit_elect(smem_u32(&s.empty[st]));
    }
    tc_commit_elect(smem_u32(&s.last));
    drain(smem_u32(&s.last), 0, p.timeout_ns);   // no product in flight when tensor memory is given back
}

__device__ __forceinline__ void copy_thread(const PrefillParams &p, PrefillShared &s, const Tile &t, int h, const CUtensorMap &qmap,
                                            const CUtensorMap &kmap, const CUtensorMap &vmap)
{
    const int hk = h / p.group;
    int issued = 0;
    for (int ch = 0; ch < t.chunks; ++ch) {
        const int st = ch & 1;
        const uint32_t bar = smem_u32(&s.full[st]), kq = smem_u32(s.KQ[st]);
        if (ch >= 2 && !mbar_wait(smem_u32(&s.empty[st]), ((ch >> 1) & 1) ^ 1, p.timeout_ns, p.status, &s.abort)) break;
        mbar_expect_tx(bar, kStageBytes);
        if ((p.debug_flags & 1) && blockIdx.x == 0 && blockIdx.y == 0) break;
        const int row = t.row0 + ch * kC;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            tma_load_2d(kq + half * 128 * 128, &kmap, hk * kD + 64 * half, row, bar);
            tma_load_2d(kq + half * 128 * 128 + kC * 128, &qmap, hk * kD + 64 * half, row, bar);
        }
        tma_load_2d(smem_u32(s.V[st]), &vmap, h * kD, row, bar);
        issued = ch + 1;
    }
    // no copy into shared memory in flight at the end
    for (int ch = max(issued - 2, 0); ch < issued; ++ch) drain(smem_u32(&s.full[ch & 1]), (ch >> 1) & 1, p.timeout_ns);
}

__global__ void __launch_bounds__(kThreads, 1)
    k_gdn_prefill(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                  const __grid_constant__ CUtensorMap vmap, const PrefillParams p)
{
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    PrefillShared &s = *reinterpret_cast<PrefillShared *>(smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u));
    const int tid = threadIdx.x, warp = tid >> 5;
    const int h = blockIdx.x, r = blockIdx.y;
    const int o0 = p.off[r], o1 = p.off[r + 1];
    if (o0 < 0 || o1 < o0 || o1 > p.n_rows) {
        if (tid == 0) atomicCAS(p.status, 0, (int32_t)W12_E_INVAL);
        return;
    }
    const Tile t{o0, o1 - o0, (o1 - o0 + kC - 1) / kC};
    if (t.n == 0) {
        // no token: the state stays what it was
        const size_t at = ((size_t)r * p.H + h) * kD * kD;
        if (p.state != p.S0)
            for (int e = tid; e < kD * kD / 4; e += kThreads)
                reinterpret_cast<float4 *>(p.state + at)[e] =
                    p.S0 ? reinterpret_cast<const float4 *>(p.S0 + at)[e] : make_float4(0.f, 0.f, 0.f, 0.f);
        return;
    }
    if (tid == 0) {
        for (int st = 0; st < 2; ++st) {
            mbar_init(smem_u32(&s.full[st]), 1);
            mbar_init(smem_u32(&s.empty[st]), 1);
            mbar_init(smem_u32(&s.ready[st]), kChunkThreads / 32);
        }
        for (unsigned long long *b : {&s.bar_kk, &s.done_k, &s.done_u, &s.done_s, &s.done_o, &s.last, &s.last_kk}) mbar_init(smem_u32(b), 1);
        for (unsigned long long *b : {&s.have_s, &s.have_x, &s.have_us, &s.have_u, &s.read_o}) mbar_init(smem_u32(b), kStateWarps);
        s.abort = 0;
        fence_mbar_init();
        prefetch_tmap(&qmap);
        prefetch_tmap(&kmap);
        prefetch_tmap(&vmap);
    }
    if (warp == 0) tmem_alloc(smem_u32(&s.tmem), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp < 8) {
        regs_inc<kRegsState>();
        state_warps(p, s, t, r, h);
    } else if (warp < 12) {
        regs_dec<kRegsChunk>();
        chunk_warps(p, s, t, h);
    } else {
        regs_dec<kRegsIssue>();
        if (warp == 12) issue_warp(p, s, t);
        if (tid == 13 * 32) copy_thread(p, s, t, h, qmap, kmap, vmap);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_dealloc(s.tmem, 512);
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
    p.n_rows = a.n_rows;
    p.timeout_ns = a.timeout_ns;
    p.status = a.status;
    p.debug_flags = a.debug_flags;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(a.H, a.n_req);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = sizeof(PrefillShared) + 1024;
    cfg.stream = static_cast<cudaStream_t>(stream);
    const cudaError_t e = cudaFuncSetAttribute(k_gdn_prefill, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)cfg.dynamicSmemBytes);
    if (e != cudaSuccess) return (int)e;
    return (int)cudaLaunchKernelEx(&cfg, k_gdn_prefill, maps[0], maps[1], maps[2], p);
}

}  // namespace w12i
