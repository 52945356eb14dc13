// Internal interface between the C-ABI host layer and the HIP kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "mxmoe.h"

namespace mxk {

// Grouped GEMM arguments (see mx_gemm.hip for the operation).
struct GemmArgs {
  const uint8_t* X;
  const uint8_t* sX;
  const uint8_t* Y;
  const uint8_t* sY;
  const int32_t* offs;
  void* C;                    // bf16 (uint16_t) or fp32 output
  int out_f32;                // 1: fp32 output, 0: bf16 (RNE)
  int64_t I, J, Kc;
  int E;
  int mode;
  int64_t ldx;                // bytes per row of X and of Y (== Kc)
  int64_t y_estride;          // mode 0: bytes between experts of Y
  int64_t sy_estride;         // mode 0: bytes between experts of sY
  int64_t ldc;                // elements per row of C
  int64_t c_estride;          // mode 1: elements between experts of C
  const int32_t* row_map;     // mode 0, optional: X row i is stored to C row row_map[i] (skipped if outside [0, c_rows))
  int64_t c_rows;
  int64_t order_mul;          // 0: the library's tile order; else workgroup slot t runs tile (t * mul + add) % grid
  int64_t order_add;
};

// gemm_rows_per_batch == 0: row-major scales [rows_total][cols/32]; > 0:
// GEMM scale layout [rows_total/R][cols/128][R][4] with R = gemm_rows_per_batch.
hipError_t launch_quant_rowwise(const uint16_t* x, int64_t rows_total, int64_t cols, uint8_t* q, uint8_t* s,
                                int64_t gemm_rows_per_batch, hipStream_t st);
// Rowwise of x[rows[r]] for r < M (index < 0 or >= src_rows: a zero row);
// scales in the GEMM layout [cols/128][M][4].
hipError_t launch_quant_rowwise_gather(const uint16_t* x, int64_t src_rows, const int32_t* rows, int64_t M,
                                       int64_t cols, uint8_t* q, uint8_t* s, hipStream_t st);
// gemm_layout == 0: s_t [batch][cols][lds]; 1: GEMM layout [batch][ldq/128][cols][4].
hipError_t launch_quant_colwise(const uint16_t* x, int64_t batch, int64_t rows, int64_t cols, uint8_t* q_t,
                                int64_t ldq, uint8_t* s_t, int64_t lds, int gemm_layout, hipStream_t st);
// Both orientations of w [E, N, K] (N % 32 == 0, K % 128 == 0, ldq % 128 == 0,
// ldq >= N): q [E, N, K] with s in GEMM layout [E][K/128][N][4]; q_t
// [E, K, ldq] with s_t in GEMM layout [E][ldq/128][K][4], zero past N.
// rows != nullptr: row n of the (batch-1) input is x[rows[n] / topk] (a zero
// row when rows[n] is negative or >= src_rows * topk): the token gather of the
// MoE dispatch.
hipError_t launch_quant_dual(const uint16_t* w, int64_t E, int64_t N, int64_t K, int64_t ldq, uint8_t* q,
                             uint8_t* s, uint8_t* q_t, uint8_t* s_t, hipStream_t st,
                             const int32_t* rows = nullptr, int64_t src_rows = 0, int topk = 1);
hipError_t launch_scales_to_gemm(const uint8_t* s, int64_t batch, int64_t rows, int64_t kb, uint8_t* out,
                                 hipStream_t st);
hipError_t launch_quant_32x32(const uint16_t* x, int64_t rows_total, int64_t cols, uint8_t* q, uint8_t* s,
                              hipStream_t st);
hipError_t launch_grouped_gemm(const GemmArgs& a, hipStream_t st);
// out[t] = bf16(sum of the k fp32 rows x[t*k .. t*k+k-1]) (see mx_topk_sum_rows).
hipError_t launch_topk_sum(const float* x, int64_t T, int k, int64_t cols, uint16_t* out, hipStream_t st);
// Routing metadata (see mx_route); ws holds route_ws_bytes(n, E) bytes.
size_t route_ws_bytes(int64_t n, int64_t E);
hipError_t launch_route(const int32_t* expert_idx, int64_t n, int64_t E, int64_t cap, int32_t* offs, int32_t* rows,
                        int32_t* pos, int32_t* status, int32_t* ws, hipStream_t st);
// status[0] = validity bitmask of the group offsets (see mx_check_offsets).
hipError_t launch_check_offsets(const int32_t* offs, int64_t E, int64_t M, int align, int32_t* status,
                                hipStream_t st);
size_t gemm_lds_bytes();

// MXFP4 (mx_fp4.hip).  Scales row-major when gemm_rows_per_batch == 0, else in
// the GEMM layout with that many rows per batch entry.
hipError_t launch_quant_rowwise_fp4(const uint16_t* x, int64_t rows_total, int64_t cols, uint8_t* q, uint8_t* s,
                                    int64_t gemm_rows_per_batch, hipStream_t st);
hipError_t launch_dequant_fp4(const uint8_t* q, const uint8_t* s, int64_t rows_total, int64_t cols, uint16_t* out,
                              int64_t gemm_rows_per_batch, hipStream_t st);
// Rows-grouped product with MXFP4 weights (see mx_fp4_gemm.hip).
struct Fp4GemmArgs {
  const uint16_t* A;          // bf16 rows [I, Kc] instead of X and sX (see fp4_gemm_takes_bf16), or null
  const uint8_t* X;           // [I, Kc] E4M3, or [I, Kc/2] E2M1 with x_fp4
  const uint8_t* sX;          // [Kc/128, I, 4]
  const uint8_t* Y;           // [E, J, Kc/2] E2M1
  const uint8_t* sY;          // [E, Kc/128, J, 4]
  const int32_t* offs;
  const int32_t* row_map;     // optional: row i goes to C row row_map[i] (dropped outside [0, c_rows))
  void* C;                    // [c_rows, J] bf16 or fp32
  int64_t I, J, Kc, c_rows;
  int E, x_fp4, out_f32;
};
hipError_t launch_fp4_gemm(const Fp4GemmArgs& a, hipStream_t st);
// Whether a product of these sizes had better quantize its bf16 rows itself.
bool fp4_gemm_takes_bf16(int64_t I, int64_t J, int64_t Kc, int64_t E);
hipError_t launch_quant_weights_fp4(const uint16_t* w, int64_t E, int64_t N, int64_t K, uint8_t* q, uint8_t* s,
                                    uint8_t* q_t, uint8_t* s_t, hipStream_t st);

constexpr int kMaxExperts = 1024;

// Gated MoE layer for a few tokens (see mx_moe.hip).
constexpr int kMoeMaxTokens = MX_MOE_MAX_TOKENS, kMoeMaxTopk = MX_MOE_MAX_TOPK;
struct MoeArgs {
  const uint16_t* x;          // bf16 [T, K]
  const int32_t* ids;         // [T, topk]
  const float* combine;       // [T, topk]
  const uint8_t* q13;         // [E, 2N, K] E4M3 or [E, 2N, K/2] E2M1
  const uint8_t* s13;         // [E, K/128, 2N, 4]
  const uint8_t* q2;          // [E, K, N] or [E, K, N/2]
  const uint8_t* s2;          // [E, N/128, K, 4]
  uint8_t* h;                 // [T * topk, N] E4M3
  uint8_t* hs;                // [T * topk, N/32]
  int32_t* meta;              // number of hit experts, then of each: expert | tokens << 16
  int2* list;                 // their tokens: row of h | token << 16, combine weight (float bits)
  uint16_t* out;              // bf16 [T, K]
  int32_t* status;            // optional: 1 when an id lies outside [0, E), else 0
  int64_t K, N;
  int T, topk, E, w_fp4;
};
hipError_t launch_moe_few_tokens(const MoeArgs& a, hipStream_t st);

// MXFP8 codes back to bf16 (mx_quant.hip); scales as launch_quant_rowwise_fp4.
hipError_t launch_dequant(const uint8_t* q, const uint8_t* s, int64_t rows_total, int64_t cols, uint16_t* out,
                          int64_t gemm_rows_per_batch, hipStream_t st);

// The router (mx_router.hip).
struct RouterArgs {
  const void* logits;         // [T, E] bf16 or fp32
  const float* bias;          // [E] or null
  int32_t* expert_idx;        // [T, k]
  float* combine;             // [T, k]
  int64_t T;
  int E, k, score, groups, topk_groups;
  int group_top2, renormalize, logits_f32;
  float scale;
};
hipError_t launch_router_fwd(const RouterArgs& a, hipStream_t st);
hipError_t launch_router_bwd(const RouterArgs& a, const float* dcombine, void* dlogits, hipStream_t st);

// The gated activation and its 8-bit checkpoint (mx_swiglu.hip).
hipError_t launch_swiglu_fwd(const uint16_t* gu, int64_t M, int64_t N, uint16_t* h, uint8_t* kept, uint8_t* kept_s,
                             hipStream_t st);
hipError_t launch_swiglu_bwd(const uint16_t* dh, const uint8_t* kept, const uint8_t* kept_s, int64_t M, int64_t N,
                             uint16_t* dgu, hipStream_t st);
struct SwigluArgs {
  const uint16_t* gu;         // [M, 2N] (forward)
  const uint16_t* dh;         // [M, N] (backward)
  const int32_t* rows;        // item of each row, or null: the row itself
  const int32_t* pos;         // row of each item, or null
  const float* combine;       // [n_items], or null: 1
  uint8_t* kept;              // [M, 2N] codes
  uint8_t* kept_s;            // [2N/128, M, 4]
  uint8_t *q, *s;             // rowwise codes and scales (GEMM layout) of h, or of dgu
  uint8_t *q_t, *s_t;         // colwise ones of w h (null: rowwise alone), or of dgu
  float* partial;             // [N/128, M] (backward), or null
  int64_t M, N, ldq, n_items;
};
int64_t swiglu_col_tiles(int64_t N);
hipError_t launch_swiglu_quantize_fwd(const SwigluArgs& a, hipStream_t st);
hipError_t launch_swiglu_quantize_bwd(const SwigluArgs& a, float* dcombine, hipStream_t st);

// The weighted sum over a token's experts (mx_combine.hip).
struct CombineArgs {
  const void* y;              // [T, k, N] bf16 or fp32
  const float* combine;       // [T, k]
  const int32_t* pos;         // [T, k] or null: negative where the item was not routed
  int64_t T, N;
  int k, y_f32;
};
hipError_t launch_combine_fwd(const CombineArgs& a, uint16_t* out, hipStream_t st);
hipError_t launch_combine_bwd(const CombineArgs& a, const uint16_t* dout, void* dy, float* dcombine, hipStream_t st);

// Record `text` as the calling thread's mx_last_error() and return `st`.
mx_status set_last_error(mx_status st, const char* text);

}  // namespace mxk
