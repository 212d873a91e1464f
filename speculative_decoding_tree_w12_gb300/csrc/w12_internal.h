// Internal declarations shared by the host ABI layer and the CUDA kernels.
#pragma once

#include <cstddef>
#include <cstdint>

#include "w12.h"

namespace w12i {

constexpr int kTileN = 128;          // output channels per W12 record
constexpr int kTileK = 64;           // input features per W12 record
constexpr int kRecBytes = 12288;     // one record: 8 KB view plane + 4 KB low nibbles
constexpr int kViewBytes = 8192;
constexpr int kMaxRows = 256;
constexpr int kMaxBudget = 512;
constexpr int kMaxPositions = 16;
constexpr int kMaxDepth = 2 * kMaxPositions + 1;   // deepest row of a spliced tree
constexpr int kCands = 16;
constexpr int kGemmSlots = 2;        // consecutive GEMMs alternate workspace slots
constexpr int kGridWords = 4096;     // GEMM-chain words: an abort word + one per GEMM of a step

// Device status word values (first condition wins).
constexpr int32_t kDevOk = 0;

// Byte layout of the caller's workspace.  Every region is 256-byte aligned.
struct WsLayout {
    size_t status;        // int32[64]: [0] status, [1] detail, [8] mismatch count (int64)
    size_t arrive;        // int32[kMaxBudget], zero between calls: the KV cache writer's arrivals (append: [0]; commit: per request)
    size_t new_len;       // int32[kMaxBudget]: the lengths that an append's last CTA writes
    size_t grid;          // uint32[kGridWords]: [0] abort word of a GEMM chain, [1 + j] CTAs done with GEMM j
    size_t counters;      // int32[kGemmSlots][max_tiles_n]: split-tile arrival counters
    size_t partial;       // float[kGemmSlots][max_ctas][2][rows8][128]
    size_t stage1_val;    // float[rows][vocab_tiles]
    size_t stage1_idx;    // int32[rows][vocab_tiles]
    size_t tree;          // tree-build scratch
    size_t total;
    int64_t max_tiles_n, max_ctas, rows8, vocab_tiles;
    int32_t rows;
};

WsLayout ws_layout(int32_t R, int64_t max_n, int64_t vocab, int32_t n_req, int num_sms);
size_t tree_ws_bytes(int32_t n_req);

// ---------------------------------------------------------------------------
// kernel launchers (defined in the .cu files); all return cudaError_t as int
// ---------------------------------------------------------------------------

struct DevWeight {
    const uint8_t *rec;
    const uint8_t *base;
    const int32_t *esc_off;
    const uint32_t *esc;
    int32_t n_tiles, k_tiles;
    int64_t n, k;
};

int launch_unpack(const DevWeight &w, uint16_t *dst, const uint16_t *cmp, int64_t *mismatch, int32_t *status,
                  void *stream);

enum GemmMode : int32_t { kModeLinear = 0, kModeHead = 1 };

struct GemmArgs {
    DevWeight w;
    const uint16_t *x;       // [R][k] row-major BF16
    int32_t R;
    int32_t mode;
    uint16_t *y;             // linear: [R][n]
    float *stage1_val;       // head: [R][n_tiles]
    int32_t *stage1_idx;
    float *partial;          // this call's slot
    int32_t *counters;       // this call's slot
    int32_t *status;
    int num_sms;
    bool pdl;                // launched as a programmatic dependent of the previous kernel
    bool qview;              // quick pass: view planes only, low mantissa bits = 0b1000 (warp-MMA path)
    int32_t debug_flags;
    uint64_t timeout_ns;
};

// The verify pass's GEMM chain in one persistent launch per up to
// chain_max_jobs() GEMMs (k_chain.cu): GEMM j + 1 reads its activations only
// after every CTA has counted itself in grid_bar[j].
struct ChainJob {
    DevWeight w;
    const uint16_t *x;       // [R][k] row-major BF16
    int32_t mode;
    uint16_t *y;             // linear: [R][n]
    float *s1_val;           // head: [R][n_tiles]
    int32_t *s1_idx;
};

struct ChainArgs {
    const ChainJob *jobs;
    int32_t n_jobs;
    int32_t R;
    float *partial;          // one partial slot (ws.partial(0))
    int32_t *counters;       // one counter slot, zero on entry
    int32_t *status;
    uint32_t *grid_bar;      // [n_jobs], zero on entry (may be null for one GEMM)
    int32_t *grid_abort;     // zero on entry
    uint64_t *trace;         // optional timing stamps (w12_debug_chain_trace)
    int num_sms;
    bool pdl;
    bool qview;
    int32_t debug_flags;
    uint64_t timeout_ns;
};

int launch_chain(const ChainArgs &a, void *stream);
int chain_max_jobs();

int launch_gemm(const GemmArgs &a, void *stream);      // warp-MMA path, R <= 64 per launch
int launch_gemm_tc(const GemmArgs &a, void *stream);   // tensor-memory path, R <= 256
// same kernel, scratch in a file-scope device array (no workspace argument)
int launch_gemm_static_scratch(const GemmArgs &a, void *stream);
int static_scratch_limits(int32_t *max_rows, int32_t *max_tiles);
int launch_argmax_stage2(const float *s1_val, const int32_t *s1_idx, int32_t R, int32_t n_tiles, int32_t *argmax,
                         float *maxlogit, bool pdl, void *stream);

struct TreeArgs {
    int32_t n_req, p_max, n_cand, conditional, budget, R;
    const int32_t *p_r_host;     // [n_req], host memory (copied into the launch parameters)
    const int32_t *root_tok;
    const int32_t *cand_tok;
    const float *cand_logp;
    int32_t *parent, *token, *req, *req_row_off;
    uint8_t *depth, *rank;
    float *score;
    void *scratch;
    int32_t *status;
};

int launch_tree_build(const TreeArgs &a, void *stream);

// certified LM head (k_cert.cu)
constexpr int kCertParts = 64;   // CTAs rescoring one row's survivors
int launch_cert_norms(const DevWeight &w, float *err, float *qnorm, void *stream);
int launch_cert_select(const uint16_t *shat, const uint16_t *h, const float *err, const float *qnorm, int32_t R,
                       int64_t V, int64_t K, int32_t *surv, int32_t *cnt, float *part_lo, void *stream);
int launch_cert_rescore(const DevWeight &w, const uint16_t *h, int32_t R, const int32_t *surv, const int32_t *cnt,
                        double *part_v, int32_t *part_i, int32_t *argmax, float *maxlogit, int32_t *cnt_out,
                        void *stream);
// recurrent-layer tree verification (k_gdn.cu)
constexpr int kGdnWy = 0, kGdnPath = 1, kGdnCommit = 2, kGdnCommitWy = 3;
constexpr int kGdnDim = 128;        // head dimension
constexpr int kGdnMaxRows = 64;     // tree rows of one request
struct GdnArgs {
    int32_t H, n_req, R;
    int num_sms;             // SMs of the device (sizes the WY kernel's grid)
    uint64_t timeout_ns;     // bounded waits of the WY kernel
    const float *S0;
    const uint16_t *q, *k, *v;
    const float *alpha, *beta;
    const int32_t *parent, *req_row_off, *acc_node;
    float *out;
    float *u;                // WY vectors [R][H][d]: written by kGdnWy when not null, read by kGdnCommitWy
    int32_t *status;
    int32_t debug_flags;     // w12_debug_set flags (bit 0: the tensor-memory WY kernel's test hook)
};
int launch_gdn(const GdnArgs &a, int mode, void *stream);

// recurrent layer over prompts (k_gdn_prefill.cu) and single tokens (k_gdn_step.cu)
struct GdnSeqArgs {
    int32_t H, Hk, n_req, n_rows;   // value heads, query/key heads
    int num_sms;
    const uint16_t *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;   // elements between rows
    const float *alpha, *beta;      // [n_rows][H]
    const int32_t *off;             // prefill: [n_req + 1]
    const float *S0;                // [n_req][H][d][d] or null (zero)
    float *state, *o;
    uint64_t timeout_ns;
    void *scratch;                  // gdn_scratch_bytes(num_sms, H, n_rows) bytes, or null
    int32_t *status;
    int32_t debug_flags;
};
size_t gdn_scratch_bytes(int num_sms, int32_t H, int32_t n_rows);
int launch_gdn_prefill(const GdnSeqArgs &a, void *stream);
int gdn_inverse_conflicts();          // see w12_debug_gdn_inverse_conflicts
int launch_gdn_step(const GdnSeqArgs &a, void *stream);

// norms around a block (k_norm.cu)
struct GdnNormArgs {
    const float *o;
    const uint16_t *z, *w;          // z may be null
    uint16_t *x;
    int64_t z_stride, x_stride;
    int32_t rows, H;
    int32_t gate_first;
    float eps;
};
int launch_gdn_norm(const GdnNormArgs &a, void *stream);
struct BlockNormArgs {
    const void *h;
    void *h_out;
    int32_t h_f32;
    const uint16_t *y, *post, *pre; // each may be null
    uint16_t *x;
    int64_t h_stride, ho_stride, y_stride, x_stride;
    int32_t rows;
    int64_t n;
    float scale, eps;
};
constexpr int64_t kMaxNormRow = 16384;
int launch_block_norm(const BlockNormArgs &a, void *stream);

// TLV splice (k_tlv.cu)
struct SpliceArgs {
    int32_t n_req, p1_max, t1_R, t2_R, R;
    const int32_t *m_host;       // [n_req], host memory (copied into the launch parameters)
    const int32_t *t1_parent, *t1_token, *t1_off;
    const uint8_t *t1_rank;
    const float *t1_score;
    const int32_t *c_tok, *c_len, *c_node;
    const int32_t *t2_parent, *t2_token, *t2_req, *t2_off;
    const uint8_t *t2_depth, *t2_rank;
    const float *t2_score;
    int32_t *parent, *token, *req, *off;
    uint8_t *depth, *rank;
    float *score;
    int32_t *status;
};
int launch_tlv_splice(const SpliceArgs &a, void *stream);

// paged 8-bit KV cache (k_kv.cu) and tree attention over it (k_attn.cu)
constexpr int kKvDim = 128;         // head dimension
constexpr int kMaxGroup = 64;       // query heads of one key/value head
struct RopeArgs {
    const float *cos, *sin;         // [max_pos][rot / 2]
    int32_t rot, adjacent, max_pos; // rot = 0: no rotation
};
struct KvArgs {
    int32_t H, bt, n_blocks, max_blocks, n_req, n_rows;
    int num_sms;
    int64_t k_stride, v_stride;     // elements between rows
    uint8_t *kc, *vc;
    float *ks, *vs;
    const int32_t *table, *len, *off;
    const int32_t *parent, *acc_node;   // commit: both set; append: null
    const uint16_t *k, *v;
    RopeArgs rope;
    int32_t *len_out, *arrive, *new_len, *status;
};
int launch_kv_write(const KvArgs &a, void *stream);

struct AttnArgs {
    int32_t H, Hq, bt, n_blocks, max_blocks, n_req, R;
    int num_sms;
    int64_t q_stride, k_stride, v_stride;
    const uint8_t *kc, *vc;
    const float *ks, *vs;
    const int32_t *table, *len, *off, *parent, *req;
    const uint8_t *depth;
    const uint16_t *q, *k, *v;
    RopeArgs rope;
    float scale;
    uint16_t *out;                  // [R][Hq][kKvDim] BF16
    void *work;                     // attn_ws_bytes
    int32_t *status;
    int32_t debug_flags;
    uint64_t timeout_ns;
};
size_t attn_ws_bytes(int32_t R, int32_t Hq, int32_t H, int32_t n_req, int num_sms);
int launch_attn(const AttnArgs &a, void *stream);
int attn_registers(int cols, int *wanted);   // registers a thread of that shape's kernel

// sampled verification (k_sample.cu)
struct SampleArgs {
    const void *logits;
    int32_t f32;
    int64_t stride, vocab;          // elements between rows; tokens
    const float *temperature;       // [n_req] or null (1)
    const float *draft_p;           // [R][vocab] or null
    int64_t draft_stride;
    const float *u_accept, *u_sample;
    int num_sms;
    void *scratch;                  // sample_scratch_bytes(R, vocab)
    int32_t R, n_req, p_max;
    const int32_t *parent, *token, *req, *off;
    int32_t *row_tok;
    float *row_logp;
    int32_t *acc_tok, *acc_len, *acc_node;   // acc_tok null: rows only
    int32_t *status;
};
int64_t sample_max_vocab();
size_t sample_scratch_bytes(int32_t R, int64_t vocab);
int launch_sample(const SampleArgs &a, void *stream);

int launch_tree_accept(const int32_t *parent, const int32_t *token, const uint8_t *depth,
                       const int32_t *req_row_off, int32_t R, int32_t n_req, int32_t p_max, const int32_t *argmax,
                       int32_t *acc_tok, int32_t *acc_len, int32_t *acc_node, bool pdl, void *stream);

}  // namespace w12i
