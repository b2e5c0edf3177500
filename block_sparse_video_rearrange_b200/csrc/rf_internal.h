// Internal declarations shared by the librf translation units (not installed).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <string>
#include <vector>

#include "rf.h"

#define RF_BLOCK 128          // query and key block rows ([API] blockShape 128 x 128)
#define RF_MAX_SEQS 32        // sequence instances one plan may hold (BNSD batch or TND seqs)
#define RF_MAX_KV_LIST 2048   // longest selectIdx row the attention kernel accepts
#define RF_MAX_NB 2048        // longest sparse region (blocks) the selection kernel accepts
#define RF_DENSE_MIN_BLOCKS 32  // [UG]: video segments below 32 blocks run dense

// Geometry of one sequence instance, passed to kernels by value.
struct RfSeqDev {
  long long row_off;    // TND: first token row of the sequence; BNSD: 0
  long long score_off;  // float offset of this sequence's [N1, nb, nb] score block in ws
  int batch_idx;        // BNSD: batch element; TND: 0
  int P, t, h, w, h8, w8;
  int A;                // aligned tokens t*h8*w8
  int S;                // sparse rows 128*nb
  int Lp;               // dense prefix rows P + promoted
  int L;                // sequence length
  int n_pb, nb, ns, k, dense;
  int order;            // rf_token_order_t of the aligned video tokens
  int qblk_off;         // first global query block
  int pool_off;         // first pooled query block (sum of nb of earlier instances)
  // Key side of the selection (block_kv rows per key block): prefix key
  // blocks, sparse key blocks, first-frame sink key blocks, ranked blocks
  // kept, and the first pooled key block.  With 128-row key blocks they are
  // n_pb, nb, ns, k and pool_off.
  int npk, nbk, nsk, kk;
  int poolk_off;
};

struct RfGeomDev {
  int n_seqs;           // instances (BNSD: batch, TND: sequences)
  int layout;           // rf_layout_t
  int n1, n2, d;
  int t_qblk;
  int max_kv;
  int block_kv;         // key/value block rows: 128, or 64 ([API] blockShape 128 x 64)
  int pooled_total;     // sum of nb over instances (query block means per head)
  int pooled_k_total;   // sum of nbk over instances (key block means per head)
  int max_nb;
  int max_nbk;
  RfSeqDev seq[RF_MAX_SEQS];
};

struct rf_plan {
  RfGeomDev g;
  rf_layout_t layout;
  rf_dtype_t dtype;
  double sparsity;
  int batch;
  int n_user_seqs;
  std::vector<rf_seq_info_t> info;  // per user sequence
  int64_t rows_total;
  int64_t ws_bytes;
  int64_t off_status, off_pq, off_pk, off_scores;
  rf_precision_t precision;
  rf_token_order_t token_order;
  int64_t off_q8, off_k8, off_qs, off_ks;  // RF_PRECISION_MIX workspace regions, else -1
  int64_t off_qx, off_kx, off_vx;          // RF_PRECISION_MXFP4 workspace regions, else -1
  int64_t off_v8, off_vexp;                // RF_PRECISION_FP8: transposed E4M3 V' and its exponents
  int64_t off_quant;                       // first precision-specific region (ws_bytes if none)
  int64_t kept_flops_upper;
};

// Workspace regions of the differential-attention calls (byte offsets), behind
// the plan's own workspace.
struct RfDiffLayout {
  int64_t v16;        // f16 copies of V' by block, [n2][t_qblk][128][d], rows past a block's end zero
  int64_t v_exp;      // int32 [n2][t_qblk]: block t of V' is v16 * 2^v_exp
  int64_t end_serve;  // what rf_diff_attn needs ends here
  int64_t stats;      // fp32 [n1][t_qblk][2][4][64]: per 64 rows -lse_1, -lse_2, delta_1, delta_2
  int64_t bits;       // query blocks that list a key block: uint32 [n1][t_qblk][words]
  int64_t dlam;       // per-block sums of dO . O_2, fp32 [n1][t_qblk]
  int64_t do_row;     // largest finite |dO| of a row, fp32 [n1][t_qblk][128] (this and the next two: fp16 plans)
  int64_t do_blk;     // {largest finite |dO|, |delta_1| and |delta_2|} of a block, float2 [n1][t_qblk]
  int64_t v_blk;      // largest finite |V| of a block, fp32 [n2][t_qblk]
  int64_t end;        // what rf_diff_attn_backward needs ends here
  int words;          // 32-bit words of one bit row: ceil(longest sequence's blocks / 32)
};
RfDiffLayout rf_diff_layout(const rf_plan* p);

// Status words at the start of the workspace.
enum { RF_STATUS_BAD_INDEX = 0, RF_STATUS_TIMEOUT = 1, RF_STATUS_WORDS = 64 };

// Error reporting (thread-local detail string).
rf_status_t rf_fail(rf_status_t st, const std::string& msg);
void rf_clear_error();  // every entry point starts with an empty detail string
rf_status_t rf_check_launch(const char* what);
rf_status_t rf_require_device();  // current device must be sm_100

// Launchers implemented in the .cu files.
rf_status_t rf_launch_rearrange(const rf_plan* p, const void* q, const void* k, const void* v,
                                void* q_r, void* k_r, void* v_r, void* ws, cudaStream_t st);
rf_status_t rf_launch_pool(const rf_plan* p, const void* q_r, const void* k_r, void* ws,
                           cudaStream_t st);
rf_status_t rf_launch_inverse(const rf_plan* p, const void* o_r, void* o, cudaStream_t st);
rf_status_t rf_launch_quantize(const rf_plan* p, const void* q_r, const void* k_r, const void* v_r,
                               void* ws, cudaStream_t st);
rf_status_t rf_launch_select(const rf_plan* p, int32_t* sel_idx, int32_t* sel_num, void* ws,
                             cudaStream_t st);
rf_status_t rf_launch_expired_wait_selftest(const rf_plan* p, void* ws, cudaStream_t st);
rf_status_t rf_launch_exp2_selftest(const float* x, float* y_poly, float* y_mufu, int64_t n,
                                    cudaStream_t st);
rf_status_t rf_launch_attn(const rf_plan* p, const void* q_r, const void* k_r, const void* v_r,
                           const int32_t* sel_idx, const int32_t* sel_num, float scale,
                           void* o_r, void* ws, cudaStream_t st);
rf_status_t rf_launch_diff_attn(const rf_plan* p, const void* q_r, const void* k_r, const void* v_r,
                                const int32_t* sel_idx, const int32_t* sel_num, const float* lambda,
                                float scale, void* o_r, float* maps, float* lse, void* ws,
                                cudaStream_t st);
rf_status_t rf_launch_diff_bwd(const rf_plan* p, const void* q_r, const void* k_r, const void* v_r,
                               const int32_t* sel_idx, const int32_t* sel_num, const float* lambda,
                               float scale, const float* maps, const float* lse, const void* do_r,
                               void* dq_r, void* dk_r, void* dv_r, float* dlambda, void* ws,
                               cudaStream_t st);
rf_status_t rf_launch_gather(const rf_plan* p, int heads, const void* x, void* x_r, bool inverse,
                             cudaStream_t st);
