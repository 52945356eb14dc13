// The gated activation between the products of an expert (gfx950), with the
// checkpoint of its input in 8 bits:
//
//   gu [M, 2N] = gate g | up u,  h = silu(g) * u
//   kept = MX8(gu), 1x32 blocks along the 2N columns: 2.06 bytes per h element
//          instead of the 4 of gu itself
//   at the kept values, s = sigmoid(g):
//   dg = dh * u * s * (1 + g (1 - s)),  du = dh * g * s
//
// Two forms.  swiglu_fwd / _bwd: bf16 in and out, the dense layer's.
// swiglu_quantize_fwd / _bwd: between two MXFP8 products of routed experts, with
// the quantization of the next product's operands in the same pass:
//   forward   q = MX8(h) along N (the down product), q_t = MX8(w h) along the rows
//             (the down weights' gradient; w: the row's combine weight)
//   backward  dgu of w dh in both orientations (the gate and up products' input
//             and weight gradients), dcombine = sum_n dh h of each row
// h, w h and dgu go from their fp32 values to E4M3, with no bf16 between.
//
// All are streaming passes, bound by HBM: bytes per h element 4 + 2 (+ 2.06) in
// swiglu_fwd, 2 + 2.06 + 4 in swiglu_bwd, 4 + 4.12 in swiglu_quantize_fwd, 2 +
// 2.06 + 4.12 in swiglu_quantize_bwd.
#include "mx_device.h"
#include "mx_kernels.h"
#include "mx_quantize.h"
#include "mx_swiglu.h"

namespace mxk {

namespace {

constexpr int kThreads = 256;

// Eight bf16 of a block spread over a quad -> codes and the block's byte.
__device__ __forceinline__ v2i quantize_quad(v4i x, uint32_t& byte) {
  byte = e8m0_from_absbits(quad_max(absmax8(x)));
  const float m = inv_scale_from_e8m0(byte == 0xFFu ? 127u : byte);
  return byte == 0xFFu ? (v2i){0x7F7F7F7F, 0x7F7F7F7F} : quant8(x, m);
}

__device__ __forceinline__ void floats8(v4i x, float* out) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    out[2 * i] = bf16lo((uint32_t)x[i]);
    out[2 * i + 1] = bf16hi((uint32_t)x[i]);
  }
}

__device__ __forceinline__ v4i pack8(const float* x) {
  return (v4i){(int)pack_bf16x2_rne(x[0], x[1]), (int)pack_bf16x2_rne(x[2], x[3]), (int)pack_bf16x2_rne(x[4], x[5]),
               (int)pack_bf16x2_rne(x[6], x[7])};
}

// Row and chunk of eight columns of chunk `i`; 32-bit division where it fits.
__device__ __forceinline__ void row_of(int64_t i, int64_t per_row, int64_t& row, int64_t& at) {
  if (i <= (int64_t)UINT32_MAX && per_row <= (int64_t)UINT32_MAX) {
    const uint32_t r = (uint32_t)i / (uint32_t)per_row;
    row = r;
    at = (uint32_t)i - r * (uint32_t)per_row;
  } else {
    row = i / per_row;
    at = i - row * per_row;
  }
}

// Gradients of eight gate and up values.
__device__ __forceinline__ void grad8(const float* dh, const float* g, const float* u, float* dg, float* du) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const Sigmoid s = sigmoid_parts(g[i]);
    dg[i] = scaled(s, s.m * fmaf(g[i], s.q, 1.f), dh[i] * u[i]);
    du[i] = scaled(s, g[i] * s.m, dh[i]);
  }
}

}  // namespace

// One thread per eight columns of h.  A DPP quad holds a block of 32.
template <bool KEEP>
__global__ __launch_bounds__(kThreads) void swiglu_fwd_kernel(const uint16_t* __restrict__ gu, int64_t chunks,
                                                              int64_t N, uint16_t* __restrict__ h,
                                                              uint8_t* __restrict__ kept, uint8_t* __restrict__ kept_s) {
  const int64_t i = wide_block() * kThreads + threadIdx.x;
  if (i >= chunks) return;
  int64_t row, c;
  row_of(i, N / 8, row, c);
  const uint16_t* src = gu + row * 2 * N + 8 * c;
  const v4i gw = __builtin_nontemporal_load((const v4i*)src);
  const v4i uw = __builtin_nontemporal_load((const v4i*)(src + N));
  float g[8], u[8], o[8];
  floats8(gw, g);
  floats8(uw, u);
#pragma unroll
  for (int j = 0; j < 8; ++j) o[j] = silu_mul(g[j], u[j]);
  *(v4i*)(h + row * N + 8 * c) = pack8(o);
  if (KEEP) {
    uint32_t gb, ub;
    const v2i gq = quantize_quad(gw, gb), uq = quantize_quad(uw, ub);
    uint8_t* dst = kept + row * 2 * N + 8 * c;
    *(v2i*)dst = gq;
    *(v2i*)(dst + N) = uq;
    if ((c & 3) == 0) {
      uint8_t* s = kept_s + row * (N / 16) + (c >> 2);
      s[0] = (uint8_t)gb;
      s[N / 32] = (uint8_t)ub;
    }
  }
}

__global__ __launch_bounds__(kThreads) void swiglu_bwd_kernel(const uint16_t* __restrict__ dh,
                                                              const uint8_t* __restrict__ kept,
                                                              const uint8_t* __restrict__ kept_s, int64_t chunks,
                                                              int64_t N, uint16_t* __restrict__ dgu) {
  const int64_t i = wide_block() * kThreads + threadIdx.x;
  if (i >= chunks) return;
  int64_t row, c;
  row_of(i, N / 8, row, c);
  const v4i dw = __builtin_nontemporal_load((const v4i*)(dh + row * N + 8 * c));
  const uint8_t* src = kept + row * 2 * N + 8 * c;
  const v2i gq = __builtin_nontemporal_load((const v2i*)src);
  const v2i uq = __builtin_nontemporal_load((const v2i*)(src + N));
  const uint8_t* s = kept_s + row * (N / 16) + (c >> 2);
  float d[8], g[8], u[8], dg[8], du[8];
  floats8(dw, d);
  values8(gq, scale_from_e8m0(s[0]), g);
  values8(uq, scale_from_e8m0(s[N / 32]), u);
  grad8(d, g, u, dg, du);
  uint16_t* dst = dgu + row * 2 * N + 8 * c;
  *(v4i*)dst = pack8(dg);
  *(v4i*)(dst + N) = pack8(du);
}

// ---------------------------------------------------------------------------
// Between two products of routed experts.  A workgroup of eight waves takes 256
// rows and 128 columns of h; wave w rows 32w..32w+31, one block of the colwise
// quantization, lane l rows 32w + 8 (l/16) + i (i < 8) and columns 8 (l%16)..: a
// quad holds a block of 32 columns, the four lanes l%16, +16, +32, +48 one of 32
// rows.  Codes of the rows go straight out, 128-byte runs; those of the columns
// through LDS, 8-byte slots swizzled so that neither side meets a bank conflict,
// and out as 256-byte runs.  Row r belongs to item rows[r]; a row with none (padding,
// behind the last group) holds anything and counts as zeros.
// ---------------------------------------------------------------------------
namespace {

constexpr int kTileRows = 256, kTileCols = 128, kTileThreads = 512;

__device__ __forceinline__ int slot16(int col, int s) { return s ^ (col >> 3 & 15); }

struct ColCodes {
  uint8_t codes[kTileCols * kTileRows];          // [column][row]
  uint8_t scales[kTileRows / 128 * kTileCols * 4];   // [128 rows][column][block]
};

// Colwise codes of the lane's 8 rows x 8 columns x[i][c] into LDS.
__device__ __forceinline__ void put_columns(ColCodes& lds, const float (&x)[8][8], int wv, int cp, int rg) {
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(x[i][c]) & 0x7FFFFFFFu);
    m = max(m, (uint32_t)__shfl_xor((int)m, 16));
    m = max(m, (uint32_t)__shfl_xor((int)m, 32));
    const uint32_t byte = e8m0_from_absbits32(m);
    float col[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) col[i] = x[i][c];
    const int k = 8 * cp + c, slot = 4 * wv + rg;
    *(v2i*)(lds.codes + k * kTileRows + 16 * slot16(k, slot >> 1) + 8 * (slot & 1)) = quant8_f32(col, byte);
    if (rg == 0) lds.scales[(wv >> 2) * (kTileCols * 4) + k * 4 + (wv & 3)] = (uint8_t)byte;
  }
}

// ... and from there to columns k0.. of q_t [., ldq] and s_t [ldq/128][cols][4].
__device__ __forceinline__ void store_columns(const ColCodes& lds, int64_t n0, int64_t k0, int64_t cols, int64_t ldq,
                                              uint8_t* __restrict__ q_t, uint8_t* __restrict__ s_t) {
  const int tid = threadIdx.x, s = tid & 15;
#pragma unroll
  for (int it = 0; it < kTileCols * 16 / kTileThreads; ++it) {
    const int k = (tid >> 4) + kTileThreads / 16 * it;
    const v4i x = *(const v4i*)(lds.codes + k * kTileRows + 16 * slot16(k, s));
    if (n0 + 16 * s < ldq) *(v4i*)(q_t + (k0 + k) * ldq + n0 + 16 * s) = x;
  }
  if (tid < 2 * kTileCols) {
    const int ch = tid / kTileCols, k = tid % kTileCols;
    if (n0 + 128 * ch < ldq)
      *(uint32_t*)(s_t + ((n0 >> 7) + ch) * cols * 4 + (k0 + k) * 4) =
          *(const uint32_t*)(lds.scales + ch * (kTileCols * 4) + k * 4);
  }
}

// Item of row r, or -1.
__device__ __forceinline__ int item_of(const SwigluArgs& a, int64_t r) {
  if (r >= a.M) return -1;
  const int64_t item = a.rows ? (int64_t)a.rows[r] : r;
  return item >= 0 && item < a.n_items ? (int)item : -1;
}

}  // namespace

template <bool TRAIN>
__global__ __launch_bounds__(kTileThreads) void swiglu_quantize_fwd_kernel(SwigluArgs a) {
  __shared__ __attribute__((aligned(16))) ColCodes lds;
  __shared__ __attribute__((aligned(16))) uint8_t srow[kTileRows * 4];
  const int tid = threadIdx.x, wv = tid >> 6, lane = tid & 63, cp = lane & 15, rg = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.y * kTileRows, k0 = (int64_t)blockIdx.x * kTileCols;
  const int r0 = 32 * wv + 8 * rg;
  int item[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) item[i] = item_of(a, n0 + r0 + i);
  v4i gw[8], uw[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    gw[i] = uw[i] = (v4i){0, 0, 0, 0};
    if (item[i] >= 0) {
      const uint16_t* src = a.gu + (n0 + r0 + i) * 2 * a.N + k0 + 8 * cp;
      gw[i] = __builtin_nontemporal_load((const v4i*)src);
      uw[i] = __builtin_nontemporal_load((const v4i*)(src + a.N));
    }
  }
  float h[8][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t r = n0 + r0 + i;
    float g[8], u[8];
    floats8(gw[i], g);
    floats8(uw[i], u);
#pragma unroll
    for (int c = 0; c < 8; ++c) h[i][c] = silu_mul(g[c], u[c]);
    const uint32_t byte = e8m0_from_absbits32(quad_max(absmax8_f32(h[i])));
    const v2i q = quant8_f32(h[i], byte);
    if (r < a.M) *(v2i*)(a.q + r * a.N + k0 + 8 * cp) = q;
    if ((cp & 3) == 0) srow[(r0 + i) * 4 + (cp >> 2)] = (uint8_t)byte;
    if (TRAIN) {
      uint32_t gb, ub;
      const v2i gq = quantize_quad(gw[i], gb), uq = quantize_quad(uw[i], ub);
      if (r < a.M) {
        uint8_t* dst = a.kept + r * 2 * a.N + k0 + 8 * cp;
        *(v2i*)dst = gq;
        *(v2i*)(dst + a.N) = uq;
        if ((cp & 3) == 0) {
          uint8_t* s = a.kept_s + r * (a.N / 16) + ((k0 + 8 * cp) >> 5);
          s[0] = (uint8_t)gb;
          s[a.N / 32] = (uint8_t)ub;
        }
      }
      const float w = item[i] < 0 ? 0.f : a.combine ? a.combine[item[i]] : 1.f;
#pragma unroll
      for (int c = 0; c < 8; ++c) h[i][c] *= w;
    }
  }
  if (TRAIN) put_columns(lds, h, wv, cp, rg);
  __syncthreads();
  if (tid < kTileRows && n0 + tid < a.M)
    *(uint32_t*)(a.s + (k0 >> 7) * a.M * 4 + (n0 + tid) * 4) = *(const uint32_t*)(srow + tid * 4);
  if (TRAIN) store_columns(lds, n0, k0, a.N, a.ldq, a.q_t, a.s_t);
}

__global__ __launch_bounds__(kTileThreads) __attribute__((amdgpu_waves_per_eu(2, 2))) void swiglu_quantize_bwd_kernel(
    SwigluArgs a) {
  __shared__ __attribute__((aligned(16))) ColCodes lds[2];
  __shared__ __attribute__((aligned(16))) uint8_t srow[2][kTileRows * 4];
  const int tid = threadIdx.x, wv = tid >> 6, lane = tid & 63, cp = lane & 15, rg = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.y * kTileRows, k0 = (int64_t)blockIdx.x * kTileCols;
  const int r0 = 32 * wv + 8 * rg;
  int item[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) item[i] = item_of(a, n0 + r0 + i);
  v4i dw[8];
  v2i gq[8], uq[8];
  uint32_t gb[8], ub[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t r = n0 + r0 + i;
    dw[i] = (v4i){0, 0, 0, 0};
    gq[i] = uq[i] = (v2i){0, 0};
    gb[i] = ub[i] = 0;
    if (item[i] >= 0) {
      dw[i] = __builtin_nontemporal_load((const v4i*)(a.dh + r * a.N + k0 + 8 * cp));
      const uint8_t* src = a.kept + r * 2 * a.N + k0 + 8 * cp;
      gq[i] = __builtin_nontemporal_load((const v2i*)src);
      uq[i] = __builtin_nontemporal_load((const v2i*)(src + a.N));
      const uint8_t* s = a.kept_s + r * (a.N / 16) + ((k0 + 8 * cp) >> 5);
      gb[i] = s[0];
      ub[i] = s[a.N / 32];
    }
  }
  float dg[8][8], du[8][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t r = n0 + r0 + i;
    const float w = item[i] < 0 ? 0.f : a.combine ? a.combine[item[i]] : 1.f;
    float d[8], g[8], u[8];
    floats8(dw[i], d);
    values8(gq[i], scale_from_e8m0(gb[i]), g);
    values8(uq[i], scale_from_e8m0(ub[i]), u);
    float dot = 0.f;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const Sigmoid s = sigmoid_parts(g[c]);
      const float e = w * d[c], gs = g[c] * s.m;
      dg[i][c] = scaled(s, s.m * fmaf(g[c], s.q, 1.f), e * u[c]);
      du[i][c] = scaled(s, gs, e);
      dot = fmaf(d[c], scaled(s, gs, u[c]), dot);
    }
    if (a.partial) {
      // over the 16 lanes of a row
      auto add = [&](int v) __attribute__((always_inline)) { dot += __int_as_float(v); };
      add(__builtin_amdgcn_mov_dpp(__float_as_int(dot), 0x128, 0xF, 0xF, false));    // row_ror:8, :4
      add(__builtin_amdgcn_mov_dpp(__float_as_int(dot), 0x124, 0xF, 0xF, false));
      add(__builtin_amdgcn_mov_dpp(__float_as_int(dot), 0x4E, 0xF, 0xF, false));     // quad [2,3,0,1], [1,0,3,2]
      add(__builtin_amdgcn_mov_dpp(__float_as_int(dot), 0xB1, 0xF, 0xF, false));
      if (cp == 0 && r < a.M) a.partial[(int64_t)blockIdx.x * a.M + r] = dot;
    }
    const uint32_t bg = e8m0_from_absbits32(quad_max(absmax8_f32(dg[i])));
    const uint32_t bu = e8m0_from_absbits32(quad_max(absmax8_f32(du[i])));
    const v2i qg = quant8_f32(dg[i], bg), qu = quant8_f32(du[i], bu);
    if (r < a.M) {
      uint8_t* dst = a.q + r * 2 * a.N + k0 + 8 * cp;
      *(v2i*)dst = qg;
      *(v2i*)(dst + a.N) = qu;
    }
    if ((cp & 3) == 0) {
      srow[0][(r0 + i) * 4 + (cp >> 2)] = (uint8_t)bg;
      srow[1][(r0 + i) * 4 + (cp >> 2)] = (uint8_t)bu;
    }
  }
  put_columns(lds[0], dg, wv, cp, rg);
  put_columns(lds[1], du, wv, cp, rg);
  __syncthreads();
  {
    const int half = tid / kTileRows, r = tid % kTileRows;
    if (n0 + r < a.M)
      *(uint32_t*)(a.s + ((half * a.N + k0) >> 7) * a.M * 4 + (n0 + r) * 4) = *(const uint32_t*)(srow[half] + r * 4);
  }
  store_columns(lds[0], n0, k0, 2 * a.N, a.ldq, a.q_t, a.s_t);
  store_columns(lds[1], n0, a.N + k0, 2 * a.N, a.ldq, a.q_t, a.s_t);
}

// dcombine[rows[r]] = sum over the column tiles of row r, in their order; items
// without a row get 0.
__global__ __launch_bounds__(kThreads) void swiglu_dcombine_kernel(SwigluArgs a, float* __restrict__ dcombine) {
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (i < a.n_items && a.pos && a.pos[i] < 0) dcombine[i] = 0.f;
  if (i >= a.M) return;
  const int item = item_of(a, i);
  if (item < 0) return;
  float sum = 0.f;
  for (int64_t t = 0; t < a.N / kTileCols; ++t) sum += a.partial[t * a.M + i];
  dcombine[item] = sum;
}

// ---------------------------------------------------------------------------
// Launchers (sizes validated by the caller).
// ---------------------------------------------------------------------------
hipError_t launch_swiglu_fwd(const uint16_t* gu, int64_t M, int64_t N, uint16_t* h, uint8_t* kept, uint8_t* kept_s,
                             hipStream_t st) {
  const int64_t chunks = M * (N / 8);
  if (chunks == 0) return hipSuccess;
  const dim3 grid = wide_grid((chunks + kThreads - 1) / kThreads);
  if (kept)
    hipLaunchKernelGGL(swiglu_fwd_kernel<true>, grid, dim3(kThreads), 0, st, gu, chunks, N, h, kept, kept_s);
  else
    hipLaunchKernelGGL(swiglu_fwd_kernel<false>, grid, dim3(kThreads), 0, st, gu, chunks, N, h, kept, kept_s);
  return hipGetLastError();
}

hipError_t launch_swiglu_bwd(const uint16_t* dh, const uint8_t* kept, const uint8_t* kept_s, int64_t M, int64_t N,
                             uint16_t* dgu, hipStream_t st) {
  const int64_t chunks = M * (N / 8);
  if (chunks == 0) return hipSuccess;
  hipLaunchKernelGGL(swiglu_bwd_kernel, wide_grid((chunks + kThreads - 1) / kThreads), dim3(kThreads), 0, st, dh, kept,
                     kept_s, chunks, N, dgu);
  return hipGetLastError();
}

int64_t swiglu_col_tiles(int64_t N) { return N / kTileCols; }

hipError_t launch_swiglu_quantize_fwd(const SwigluArgs& a, hipStream_t st) {
  const int64_t rows = a.q_t ? a.ldq : a.M;
  if (rows == 0 || a.N == 0) return hipSuccess;
  const dim3 grid((unsigned)(a.N / kTileCols), (unsigned)((rows + kTileRows - 1) / kTileRows));
  if (a.q_t) hipLaunchKernelGGL(swiglu_quantize_fwd_kernel<true>, grid, dim3(kTileThreads), 0, st, a);
  else hipLaunchKernelGGL(swiglu_quantize_fwd_kernel<false>, grid, dim3(kTileThreads), 0, st, a);
  return hipGetLastError();
}

hipError_t launch_swiglu_quantize_bwd(const SwigluArgs& a, float* dcombine, hipStream_t st) {
  if (a.ldq > 0 && a.N > 0) {
    const dim3 grid((unsigned)(a.N / kTileCols), (unsigned)((a.ldq + kTileRows - 1) / kTileRows));
    hipLaunchKernelGGL(swiglu_quantize_bwd_kernel, grid, dim3(kTileThreads), 0, st, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const int64_t n = a.M > a.n_items ? a.M : a.n_items;
  if (!dcombine || n == 0) return hipSuccess;
  hipLaunchKernelGGL(swiglu_dcombine_kernel, dim3((unsigned)((n + kThreads - 1) / kThreads)), dim3(kThreads), 0, st, a,
                     dcombine);
  return hipGetLastError();
}

}  // namespace mxk
