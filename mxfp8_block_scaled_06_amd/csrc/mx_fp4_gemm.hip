// Grouped product with MXFP4 weights (gfx950):
//
//   C[i, j] = sum_k X[i, k] * Y[e][j, k] * 2^(sX[i, k/32] + sY[e][j, k/32] - 254)
//
// for the rows i of expert e, X in MXFP8 (E4M3) or MXFP4 (E2M1), Y in MXFP4,
// accumulated in fp32 by the block-scaled matrix instructions, which take the
// E8M0 bytes as they are and each operand in its own format.
//
// Operand layouts of v_mfma_scale_f32_16x16x128_f8f6f4, checked on the card
// for both formats and the mixed product: lane l holds row l%16 of its
// operand, group g = l/16.  E2M1: the 16 bytes of elements 32g .. 32g+31.
// E4M3: the 16-byte pieces g and g+4 of the 128 elements.  The scale byte of
// lane l covers block g.  Lane l's four accumulators are column l%16, rows
// 4g .. 4g+3.  (32x32x64: l%32, g = l/32, pieces g and g+2, rows
// 8(r/4) + 4g + r%4.)  Y is the first operand, so a lane holds runs of four
// output columns of one output row.
#include "mx_device.h"
#include "mx_kernels.h"
#include "mx_rows_tiles.h"

namespace mxk {

typedef float v4f __attribute__((ext_vector_type(4)));

constexpr int kFmtE4M3 = 0, kFmtE2M1 = 4;      // the instruction's operand formats

// ---------------------------------------------------------------------------
// Few rows per expert: the product streams the weights once and is bound by
// that.  A workgroup of 8 waves takes 64 rows x 32 columns and splits the
// contraction: wave w multiplies a contiguous eighth of the 128-element
// chunks straight from global memory (each weight byte is used by one
// workgroup row only, so LDS would add a copy and a barrier), and the partial
// sums meet in LDS, added in wave order.
// ---------------------------------------------------------------------------
constexpr int kSmBM = 64, kSmBN = 32, kSmWaves = 8;
constexpr int kSmCT = kSmBM / 16, kSmRT = kSmBN / 16;

template <int XF, bool OUT_F32>
__global__ __launch_bounds__(kSmWaves * 64) void fp4_rows_small_kernel(Fp4GemmArgs a) {
  __shared__ int s_offs[kMaxExperts], s_pref[kMaxExperts], s_total;
  __shared__ v4f part[kSmWaves][kSmRT * kSmCT][64];
  const rows::Tile t =
      rows::find_tile<kSmBM, kSmBN, kSmWaves * 64>(a.offs, a.E, a.I, a.J, s_offs, s_pref, &s_total);
  if (!t.valid) return;
  const int tid = threadIdx.x, lane = tid & 63, wv = rows::uni32(tid >> 6);
  const int l16 = lane & 15, g = lane >> 4;
  const int e = rows::uni32(t.e);
  const int64_t i0 = rows::uni64(t.i0), i_end = rows::uni64(t.i_end), j0 = rows::uni64(t.j0);
  const int nx = (int)min((int64_t)kSmBM, i_end - i0);
  const int ny = (int)min((int64_t)kSmBN, a.J - j0);
  const int64_t ldx = XF == kFmtE4M3 ? a.Kc : a.Kc / 2, ldy = a.Kc / 2;
  const __amdgpu_buffer_rsrc_t rx = rows::rsrc(a.X + i0 * ldx, nx * ldx);
  const __amdgpu_buffer_rsrc_t ry = rows::rsrc(a.Y + ((int64_t)e * a.J + j0) * ldy, ny * ldy);
  const uint8_t* sx = a.sX + i0 * 4 + g;
  const uint8_t* sy = a.sY + (int64_t)e * a.J * (a.Kc / 32) + j0 * 4 + g;
  const int nch = (int)(a.Kc / 128), per = (nch + kSmWaves - 1) / kSmWaves;
  const int nct = (nx + 15) / 16;     // column tiles that hold rows of the group
  v4f acc[kSmRT][kSmCT];
#pragma unroll
  for (int r = 0; r < kSmRT; ++r)
#pragma unroll
    for (int c = 0; c < kSmCT; ++c) acc[r][c] = (v4f){0.f, 0.f, 0.f, 0.f};
  const int c_end = min((wv + 1) * per, nch);
  for (int ch = wv * per; ch < c_end; ++ch) {
    v8i y[kSmRT];
    int ys[kSmRT];
#pragma unroll
    for (int r = 0; r < kSmRT; ++r) {
      const int row = 16 * r + l16;
      const v4i w = __builtin_amdgcn_raw_buffer_load_b128(ry, (int)(row * ldy) + ch * 64 + 16 * g, 0, 0);
      y[r] = (v8i){w[0], w[1], w[2], w[3], 0, 0, 0, 0};
      ys[r] = sy[(ch * a.J + min(row, ny - 1)) * 4];      // rows past the end are read as zeros and never stored
    }
#pragma unroll
    for (int c = 0; c < kSmCT; ++c) {
      if (c >= nct) continue;
      const int row = 16 * c + l16;
      v8i x;
      if (XF == kFmtE4M3) {
        const v4i p = __builtin_amdgcn_raw_buffer_load_b128(rx, (int)(row * ldx) + ch * 128 + 16 * g, 0, 0);
        const v4i q = __builtin_amdgcn_raw_buffer_load_b128(rx, (int)(row * ldx) + ch * 128 + 64 + 16 * g, 0, 0);
        x = (v8i){p[0], p[1], p[2], p[3], q[0], q[1], q[2], q[3]};
      } else {
        const v4i p = __builtin_amdgcn_raw_buffer_load_b128(rx, (int)(row * ldx) + ch * 64 + 16 * g, 0, 0);
        x = (v8i){p[0], p[1], p[2], p[3], 0, 0, 0, 0};
      }
      const int xs = sx[(ch * a.I + min(row, nx - 1)) * 4];
#pragma unroll
      for (int r = 0; r < kSmRT; ++r)
        acc[r][c] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(y[r], x, acc[r][c], kFmtE2M1, XF, 0, ys[r], 0, xs);
    }
  }
#pragma unroll
  for (int r = 0; r < kSmRT; ++r)
#pragma unroll
    for (int c = 0; c < kSmCT; ++c) part[wv][r * kSmCT + c][lane] = acc[r][c];
  __syncthreads();
  // one run of four output columns per thread
  static_assert(kSmRT * kSmCT * 64 == kSmWaves * 64, "one run per thread");
  const int rt = wv / kSmCT, ct = wv % kSmCT;
  v4f s = part[0][wv][lane];
#pragma unroll
  for (int w = 1; w < kSmWaves; ++w) s += part[w][wv][lane];
  const int64_t i = i0 + 16 * ct + l16, j = j0 + 16 * rt + 4 * g;
  if (i >= i_end || j >= a.J) return;
  const int64_t dst = a.row_map ? (int64_t)a.row_map[i] : i;
  if (dst < 0 || dst >= a.c_rows) return;
  if (OUT_F32) {
    *(v4f*)((float*)a.C + dst * a.J + j) = s;
  } else {
    *(v2i*)((uint16_t*)a.C + dst * a.J + j) =
        (v2i){(int)pack_bf16x2_rne(s[0], s[1]), (int)pack_bf16x2_rne(s[2], s[3])};
  }
}

hipError_t launch_fp4_gemm(const Fp4GemmArgs& a, hipStream_t st) {
  if (a.I == 0 || a.J == 0) return hipSuccess;
  const dim3 grid((unsigned)rows::grid<kSmBM, kSmBN>(a.I, a.J, a.E)), block(kSmWaves * 64);
  if (a.x_fp4) {
    if (a.out_f32) hipLaunchKernelGGL((fp4_rows_small_kernel<kFmtE2M1, true>), grid, block, 0, st, a);
    else hipLaunchKernelGGL((fp4_rows_small_kernel<kFmtE2M1, false>), grid, block, 0, st, a);
  } else {
    if (a.out_f32) hipLaunchKernelGGL((fp4_rows_small_kernel<kFmtE4M3, true>), grid, block, 0, st, a);
    else hipLaunchKernelGGL((fp4_rows_small_kernel<kFmtE4M3, false>), grid, block, 0, st, a);
  }
  return hipGetLastError();
}

}  // namespace mxk
