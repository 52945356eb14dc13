// Grouped product with MXFP4 weights (gfx950):
//
//   C[i, j] = sum_k X[i, k] * Y[e][j, k] * 2^(sX[i, k/32] + sY[e][j, k/32] - 254)
//
// for the rows i of expert e, X in MXFP8 (E4M3) or MXFP4 (E2M1), Y in MXFP4,
// accumulated in fp32 by the block-scaled matrix instructions, which take the
// E8M0 bytes as they are and each operand in its own format.  With E4M3 rows the
// instruction drops the low bits of products far below the largest that it adds:
// at most 1.6e-4 of the sum of magnitudes was seen, E2M1 rows gave exact sums.
//
// Operand layouts of v_mfma_scale_f32_16x16x128_f8f6f4, checked on the card
// for both formats and the mixed product: lane l holds row l%16 of its
// operand, group g = l/16.  E2M1: the 16 bytes of elements 32g .. 32g+31.
// E4M3: the 16-byte pieces g and g+4 of the 128 elements.  The scale byte of
// lane l covers block g.  Lane l's four accumulators are column l%16, rows
// 4g .. 4g+3.  (32x32x64: l%32, g = l/32, pieces g and g+2, rows
// 8(r/4) + 4g + r%4.)  Y is the first operand, so a lane holds runs of four
// output columns of one output row.
#include <algorithm>
#include <type_traits>

#include "mx_device.h"
#include "mx_kernels.h"
#include "mx_quantize.h"
#include "mx_rows_tiles.h"

namespace mxk {

typedef float v4f __attribute__((ext_vector_type(4)));

constexpr int kFmtE4M3 = 0, kFmtE2M1 = 4;      // the instruction's operand formats

// ---------------------------------------------------------------------------
// Few output tiles: the product streams the weights once and is bound by that,
// and 256 x 256 tiles would leave CUs idle.  A workgroup of 8 waves takes 64
// rows x 32 columns and splits the contraction: each wave multiplies its run of
// 256-element units (whole 128-byte lines of the weight rows) straight from
// memory, and the partial sums meet in LDS, added in wave order.
// ---------------------------------------------------------------------------
constexpr int kSmBM = 64, kSmBN = 32, kSmWaves = 8;
constexpr int kSmCT = kSmBM / 16, kSmRT = kSmBN / 16;

// 16 bytes of codes of four 16-byte pieces of bf16 values, in the lane's operand
// layout, and its scale byte: the codes and bytes of the row quantizers.  E2M1:
// the pieces are block g.  E4M3: two pieces of block g/2 and two of 2 + g/2, each
// shared with the lanes of group g ^ 1.
template <int XF>
__device__ __forceinline__ void quantize_operand(const v4i w[4], int g, v4i x[2], int& scale) {
  us2 m[2] = {__builtin_elementwise_max(absmax8x2(w[0]), absmax8x2(w[1])),
              __builtin_elementwise_max(absmax8x2(w[2]), absmax8x2(w[3]))};
  if (XF == kFmtE4M3) {
    uint32_t byte[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t v = max(m[i][0], m[i][1]);
      const auto o = __builtin_amdgcn_permlane16_swap(v, v, false, false);      // groups 0 0 2 2 and 1 1 3 3
      byte[i] = e8m0_from_absbits(max(o[0], o[1]));
      const uint32_t most = ((byte[i] + 8u) << 7 | 0x60u) * 0x10001u;
      const v2i lo = quantize8(w[2 * i], byte[i], most), hi = quantize8(w[2 * i + 1], byte[i], most);
      const bool nan = byte[i] == 0xFFu;
      x[i] = nan ? (v4i){0x7F7F7F7F, 0x7F7F7F7F, 0x7F7F7F7F, 0x7F7F7F7F} : (v4i){lo[0], lo[1], hi[0], hi[1]};
    }
    // block g's byte: blocks 0 0 2 2 of the four groups, and 1 1 3 3
    const auto o = __builtin_amdgcn_permlane32_swap(byte[0], byte[1], false, false);
    scale = (int)(g & 1 ? o[1] : o[0]);
  } else {
    const us2 all = __builtin_elementwise_max(m[0], m[1]);
    const uint32_t byte = e8m0_fp4_from_absbits(max(all[0], all[1]));
#pragma unroll
    for (int i = 0; i < 4; ++i) x[0][i] = (int)quant8_fp4(w[i], byte);
    scale = (int)byte;
  }
}

// BF16: the rows are a.A, quantized to XF here.
template <int XF, bool OUT_F32, bool BF16>
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
  const __amdgpu_buffer_rsrc_t rx = BF16 ? rows::rsrc(a.A + i0 * a.Kc, nx * a.Kc * 2) : rows::rsrc(a.X + i0 * ldx, nx * ldx);
  const __amdgpu_buffer_rsrc_t ry = rows::rsrc(a.Y + ((int64_t)e * a.J + j0) * ldy, ny * ldy);
  const uint8_t* sx = a.sX + i0 * 4 + g;
  const uint8_t* sy = a.sY + (int64_t)e * a.J * (a.Kc / 32) + j0 * 4 + g;
  const int nch = (int)(a.Kc / 128), units = (nch + 1) / 2;
  const int nct = (nx + 15) / 16;     // column tiles that hold rows of the group
  v4f acc[kSmRT][kSmCT];
#pragma unroll
  for (int r = 0; r < kSmRT; ++r)
#pragma unroll
    for (int c = 0; c < kSmCT; ++c) acc[r][c] = (v4f){0.f, 0.f, 0.f, 0.f};
  const int end = units * (wv + 1) / kSmWaves;
  for (int u = units * wv / kSmWaves; u < end; ++u) {
    v4i y[kSmRT][2], x[kSmCT][2][BF16 ? 4 : XF == kFmtE4M3 ? 2 : 1];
    int ys[kSmRT][2], xs[kSmCT][2];
    // a line's second chunk past the end is not multiplied
    const int ch[2] = {2 * u, min(2 * u + 1, nch - 1)};
#pragma unroll
    for (int r = 0; r < kSmRT; ++r) {
      const int row = 16 * r + l16;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        y[r][i] = __builtin_amdgcn_raw_buffer_load_b128(ry, (int)(row * ldy) + u * 128 + 64 * i + 16 * g, 0, 0);
        ys[r][i] = sy[(ch[i] * a.J + min(row, ny - 1)) * 4];      // rows past the end are read as zeros and never stored
      }
    }
#pragma unroll
    for (int c = 0; c < kSmCT; ++c) {
      if (c >= nct) continue;
      const int row = 16 * c + l16;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if constexpr (BF16) {
          const int o = (int)(row * a.Kc + ch[i] * 128) * 2;
#pragma unroll
          for (int k = 0; k < 4; ++k)
            x[c][i][k] = __builtin_amdgcn_raw_buffer_load_b128(
                rx, o + (XF == kFmtE4M3 ? 32 * g + 16 * (k & 1) + 128 * (k >> 1) : 64 * g + 16 * k), 0, 0);
          continue;
        } else if constexpr (XF == kFmtE4M3) {
          x[c][i][0] = __builtin_amdgcn_raw_buffer_load_b128(rx, (int)(row * ldx) + ch[i] * 128 + 16 * g, 0, 0);
          x[c][i][XF == kFmtE4M3] =
              __builtin_amdgcn_raw_buffer_load_b128(rx, (int)(row * ldx) + ch[i] * 128 + 64 + 16 * g, 0, 0);
        } else {
          x[c][i][0] = __builtin_amdgcn_raw_buffer_load_b128(rx, (int)(row * ldx) + ch[i] * 64 + 16 * g, 0, 0);
        }
        xs[c][i] = sx[(ch[i] * a.I + min(row, nx - 1)) * 4];
      }
    }
#pragma unroll
    for (int c = 0; c < kSmCT; ++c) {
      if (c >= nct) continue;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (2 * u + i >= nch) continue;
        if constexpr (BF16) {
          v4i codes[2];
          quantize_operand<XF>(x[c][i], g, codes, xs[c][i]);
          x[c][i][0] = codes[0];
          x[c][i][1] = codes[1];
        }
        v8i xv;
        if (XF == kFmtE4M3) xv = __builtin_shufflevector(x[c][i][0], x[c][i][XF == kFmtE4M3], 0, 1, 2, 3, 4, 5, 6, 7);
        else xv = __builtin_shufflevector(x[c][i][0], x[c][i][0], 0, 1, 2, 3, -1, -1, -1, -1);
#pragma unroll
        for (int r = 0; r < kSmRT; ++r)
          acc[r][c] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
              __builtin_shufflevector(y[r][i], y[r][i], 0, 1, 2, 3, -1, -1, -1, -1), xv, acc[r][c], kFmtE2M1, XF, 0,
              ys[r][i], 0, xs[c][i]);
      }
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

// ---------------------------------------------------------------------------
// Many rows per expert: 256 x 256 output tiles, 8 waves (two per SIMD) of
// 128 x 64, 128 fp32 accumulators per lane.  A stage is 128 contraction
// elements; its codes and scales move from memory into LDS by direct loads
// (no registers between), kBufs stages deep.  Waves 0..3, one per SIMD, issue
// all of the loads, so that a wave held up by a full address queue leaves its
// SIMD's matrix core to the other one; waves 4..7 only read LDS and multiply.
// A stage has two 64-element windows.  Each wave reads the next window's
// fragments while the current one's matrix instructions run, and there is one
// barrier per stage, at the start of its second window: by then every wave has
// the stage's last fragments in registers, so its buffer can take the stage
// kBufs later, and the next stage has landed.  That stage's loads are spread
// over this window and the first one of the next stage: half of them in each
// took 605-614 us where all in the first took 627-632 (16384 x 8192 x 5120
// over 16 experts, MXFP8 activations), 409 against 424 on Zipf routing.
//
// What bounds it: the power of moving operands.  On constant data the same
// launch (dense 16384 x 8192 x 5120, MXFP8) takes 400 us instead of 494, and
// 366 when no operand moves.  MXFP4 rows arrive as 64-byte halves of lines;
// stages of 256 elements (whole lines) leave room for two buffers instead of
// four and were slower on ragged groups (445 against 430 us).
// ---------------------------------------------------------------------------
typedef __attribute__((address_space(3))) void lds_ptr;

constexpr int kBM = 256, kBN = 256, kThreads = 512;
constexpr int kOutPitch = kBN * 2 + 16;        // bytes per staged bf16 output row (+16: spreads banks)

template <int XF>
struct Stage {
  static constexpr int kXRow = XF == kFmtE4M3 ? 128 : 64, kYRow = 64;   // code bytes per row
  static constexpr int kX = kBM * kXRow, kY = kBN * kYRow, kScale = 256 * 4;
  static constexpr int kBytes = kX + kY + 2 * kScale;
  // the deepest that fits in 160 KiB with the epilogue's tile inside it
  static constexpr int kBufs = XF == kFmtE4M3 ? 3 : 4;
  static constexpr int kXLoads = kX / 4096, kYLoads = kY / 4096;        // one-KiB loads per loading wave
  static constexpr int kLoads = kXLoads + kYLoads + 2;                  // and the scales of its 64 rows, twice 256 B
  static constexpr int kFirst = kLoads / 2;                             // of them in the stage's second window
};
static_assert(kBM * kOutPitch <= Stage<kFmtE4M3>::kBytes * 3 && kBM * kOutPitch <= Stage<kFmtE2M1>::kBytes * 4, "epilogue");

// 16-byte slot of a piece in its LDS row: the lanes that read one logical
// piece of consecutive rows spread over all banks (rows of 128 or 64 bytes).
template <int ROW>
__device__ __forceinline__ int swz(int row) {
  return ROW == 128 ? (row >> 1) & 7 : (row >> 2) & 3;
}

// One stage's loads: descriptors and the LDS buffer.
struct Dma {
  __amdgpu_buffer_rsrc_t rx, ry, rsx, rsy;
  uint8_t* st;
};

struct Frag {
  v8i v;
  int s;      // the row's scale dword, shifted so that bytes 0 and 2 are this lane's blocks of windows 0 and 1
};

template <int M, int N, class F>
__device__ __forceinline__ void static_for(F&& f) {
  if constexpr (M < N) {
    f(std::integral_constant<int, M>{});
    static_for<M + 1, N>(f);
  }
}

template <int XF, bool OUT_F32>
__global__ __launch_bounds__(kThreads, 1) void fp4_rows_kernel(Fp4GemmArgs a) {
  using S = Stage<XF>;
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
  int* s_offs = (int*)smem;
  const rows::Tile t = rows::find_tile<kBM, kBN, kThreads>(a.offs, a.E, a.I, a.J, s_offs, s_offs + kMaxExperts,
                                                           s_offs + 2 * kMaxExperts);
  if (!t.valid) return;
  __syncthreads();      // the scheduler's arrays make room for the first stages
  const int tid = threadIdx.x, lane = tid & 63, wv = rows::uni32(tid >> 6);
  const int iw = wv >> 2, jw = wv & 3;        // the wave's 128 x 64 block
  const int half = lane >> 5, l32 = lane & 31;
  const int e = rows::uni32(t.e);
  const int64_t i0 = rows::uni64(t.i0), i_end = rows::uni64(t.i_end), j0 = rows::uni64(t.j0);
  const int rows_x = (int)min((int64_t)kBM, i_end - i0), rows_y = (int)min((int64_t)kBN, a.J - j0);
  const int ns = (int)(a.Kc / 128);
  const int64_t ldx = XF == kFmtE4M3 ? a.Kc : a.Kc / 2, ldy = a.Kc / 2;
  const uint8_t* xb = a.X + i0 * ldx;
  const uint8_t* yb = a.Y + ((int64_t)e * a.J + j0) * ldy;
  const uint8_t* sxb = a.sX + i0 * 4;
  const uint8_t* syb = a.sY + (int64_t)e * a.J * (a.Kc / 32) + j0 * 4;

  // this lane's part of a one-KiB load: rows of 128 bytes (8 lanes each) or 64
  constexpr int kXLanes = S::kXRow / 16, kYLanes = S::kYRow / 16;
  const int lw = wv & 3;
  int xoff, yoff;      // byte offsets of load 0; load u is u * (64 / lanes per row) rows on, same slot
  {
    const int xr = lw * 64 + lane / kXLanes, yr = lw * 64 + lane / kYLanes;
    xoff = xr * (int)ldx + (((lane % kXLanes) ^ swz<S::kXRow>(xr)) << 4);
    yoff = yr * (int)ldy + (((lane % kYLanes) ^ swz<S::kYRow>(yr)) << 4);
  }
  // 128-byte rows: load u covers rows 8u.., whose swizzle repeats every 16 rows
  const int xoff1 = XF == kFmtE4M3
                        ? (lw * 64 + 8 + lane / kXLanes) * (int)ldx +
                              (((lane % kXLanes) ^ swz<S::kXRow>(lw * 64 + 8 + lane / kXLanes)) << 4)
                        : 0;
  // Stages at or past ns get empty ranges: no data moves, but the loads are
  // issued, so that the counts that the waits go by are the same throughout.
  auto make_dma = [&](int buf, int kt) __attribute__((always_inline)) {
    Dma d;
    d.st = smem + buf * S::kBytes;
    const bool live = kt < ns;
    const int64_t kx = (int64_t)kt * S::kXRow, ky = (int64_t)kt * S::kYRow;
    d.rx = rows::rsrc(xb + kx, live ? rows_x * ldx - kx : 0);
    d.ry = rows::rsrc(yb + ky, live ? rows_y * ldy - ky : 0);
    d.rsx = rows::rsrc(sxb + (int64_t)kt * a.I * 4, live ? (a.I - i0) * 4 : 0);
    d.rsy = rows::rsrc(syb + (int64_t)kt * a.J * 4, live ? (a.J - j0) * 4 : 0);
    return d;
  };
  auto issue = [&](auto nc, const Dma& d) __attribute__((always_inline)) {
    constexpr int n = decltype(nc)::value;
    if constexpr (n < S::kXLoads) {
      const int vo = XF == kFmtE4M3 ? ((n & 1) ? xoff1 : xoff) + (n >> 1) * 16 * (int)ldx : xoff + n * 16 * (int)ldx;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(d.rx, (lds_ptr*)(d.st + (lw * S::kXLoads + n) * 1024), 16, vo, 0, 0, 0);
    } else if constexpr (n < S::kXLoads + S::kYLoads) {
      constexpr int u = n - S::kXLoads;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(d.ry, (lds_ptr*)(d.st + S::kX + (lw * S::kYLoads + u) * 1024), 16,
                                               yoff + u * 16 * (int)ldy, 0, 0, 0);
    } else if constexpr (n == S::kXLoads + S::kYLoads) {
      __builtin_amdgcn_raw_ptr_buffer_load_lds(d.rsx, (lds_ptr*)(d.st + S::kX + S::kY + lw * 256), 4,
                                               (lw * 64 + lane) * 4, 0, 0, 0);
    } else {
      __builtin_amdgcn_raw_ptr_buffer_load_lds(d.rsy, (lds_ptr*)(d.st + S::kX + S::kY + S::kScale + lw * 256), 4,
                                               (lw * 64 + lane) * 4, 0, 0, 0);
    }
  };

  v16f acc[2][4];
#pragma unroll
  for (int y = 0; y < 2; ++y)
#pragma unroll
    for (int x = 0; x < 4; ++x) acc[y][x] = (v16f){};

  // this lane's fragment addresses inside a stage (the swizzle goes by l32 alone)
  const int xrow = iw * 128 + l32, yrow = jw * 64 + l32;
  int xo[2][2], yo[2];
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    yo[w] = S::kX + yrow * S::kYRow + (((2 * w + half) ^ swz<S::kYRow>(l32)) << 4);
#pragma unroll
    for (int c = 0; c < 2; ++c)
      xo[w][c] = xrow * S::kXRow +
                 (((XF == kFmtE4M3 ? 4 * w + half + 2 * c : 2 * w + half) ^ swz<S::kXRow>(l32)) << 4);
  }
  const int sxo = S::kX + S::kY + xrow * 4, syo = S::kX + S::kY + S::kScale + yrow * 4;
  auto read_x = [&](const uint8_t* st, int w, int sub, Frag& f) __attribute__((always_inline)) {
    const v4i p = *(const v4i*)(st + xo[w][0] + sub * 32 * S::kXRow);
    if (XF == kFmtE4M3) {
      const v4i q = *(const v4i*)(st + xo[w][1] + sub * 32 * S::kXRow);
      f.v = (v8i){p[0], p[1], p[2], p[3], q[0], q[1], q[2], q[3]};
    } else {
      f.v = __builtin_shufflevector(p, p, 0, 1, 2, 3, -1, -1, -1, -1);
    }
    if (w == 0) f.s = *(const int*)(st + sxo + sub * 32 * 4) >> (8 * half);
  };
  auto read_y = [&](const uint8_t* st, int w, int sub, Frag& f) __attribute__((always_inline)) {
    const v4i p = *(const v4i*)(st + yo[w] + sub * 32 * S::kYRow);
    f.v = __builtin_shufflevector(p, p, 0, 1, 2, 3, -1, -1, -1, -1);
    if (w == 0) f.s = *(const int*)(st + syo + sub * 32 * 4) >> (8 * half);
  };

  // X sub-tiles qx = 0..3 in FX[0..2] and FX[3 + window] (the last one alternates
  // so that its refill does not wait for the window's last instruction), Y
  // sub-tiles in FY[window].
  Frag FX[5], FY[2][2];
  // Window W: its eight matrix instructions, the reads of the other window of
  // `src`, and this wave's part of the loads of `pend`.
  auto window = [&](auto w_c, auto nxs_c, auto loads_c, const uint8_t* src, const Dma& pend)
                    __attribute__((always_inline)) {
    constexpr int W = decltype(w_c)::value, NW = W ^ 1, NXS = decltype(nxs_c)::value;
    constexpr bool LOADS = decltype(loads_c)::value;
    constexpr int kFrom = W == 1 ? 0 : S::kFirst, kTo = W == 1 ? S::kFirst : S::kLoads;
    static_for<0, 8>([&](auto mc) {
      constexpr int m = decltype(mc)::value, qx = m >> 1, qy = m & 1, xi = qx < 3 ? qx : 3 + W;
      if constexpr (qx < NXS)
        acc[qy][qx] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(FY[W][qy].v, FX[xi].v, acc[qy][qx], kFmtE2M1, XF,
                                                                      2 * W, FY[W][qy].s, 2 * W, FX[xi].s);
      if constexpr (LOADS) {
        // spread over the window's instructions
        static_for<kFrom + m * (kTo - kFrom) / 8, kFrom + (m + 1) * (kTo - kFrom) / 8>([&](auto nc) { issue(nc, pend); });
      }
      if constexpr (NXS > 0) {
        if constexpr (m < 2) {
          read_y(src, NW, m, FY[NW][m]);
          if constexpr (W == 0) FY[NW][m].s = FY[W][m].s;
        }
        if constexpr (m == 0 && NXS > 3) {
          read_x(src, NW, 3, FX[3 + NW]);
          if constexpr (W == 0) FX[3 + NW].s = FX[3 + W].s;
        }
        if constexpr (m == 1 || m == 3 || m == 5) {
          if constexpr ((m >> 1) < NXS) read_x(src, NW, m >> 1, FX[m >> 1]);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    });
  };
  auto run = [&](auto nxs_c, auto dma_c) __attribute__((always_inline)) {
    constexpr int NXS = decltype(nxs_c)::value;
    constexpr bool DMA = decltype(dma_c)::value;
    if constexpr (DMA) {
      static_for<0, S::kBufs>([&](auto bc) {
        const Dma d = make_dma(decltype(bc)::value, decltype(bc)::value);
        static_for<0, decltype(bc)::value == S::kBufs - 1 ? S::kFirst : S::kLoads>([&](auto nc) { issue(nc, d); });
      });
      // stage 0 has landed
      asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(S::kLoads * (S::kBufs - 2) + S::kFirst) : "memory");
    } else {
      asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    }
    if constexpr (NXS > 0) {
      read_y(smem, 0, 0, FY[0][0]);
      read_y(smem, 0, 1, FY[0][1]);
    }
    static_for<0, 4>([&](auto fc) {
      constexpr int f = decltype(fc)::value;
      if constexpr (f < NXS) read_x(smem, 0, f, FX[f]);
    });
    int buf = 0, last = S::kBufs - 1;      // buffers of stages kt and kt - 1
    for (int kt = 0; kt < ns; ++kt) {
      const int nbuf = buf + 1 == S::kBufs ? 0 : buf + 1;
      const uint8_t* cs = smem + buf * S::kBytes;
      const uint8_t* nst = smem + nbuf * S::kBytes;
      const Dma rest = make_dma(last, kt + S::kBufs - 1);
      window(std::integral_constant<int, 0>{}, nxs_c, dma_c, cs, rest);
      // stage kt+1 has landed; every wave is done reading this buffer
      if constexpr (DMA)
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(S::kLoads * (S::kBufs - 2)) : "memory");
      else
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
      const Dma pend = make_dma(buf, kt + S::kBufs);
      window(std::integral_constant<int, 1>{}, nxs_c, dma_c, nst, pend);
      last = buf;
      buf = nbuf;
    }
  };
  // 32-row sub-tiles of this wave that hold rows of the group: a partial last
  // M-tile multiplies no others
  const int nxs = min(max((rows_x - iw * 128 + 31) >> 5, 0), 4);
  auto by_nxs = [&](auto dma_c) __attribute__((always_inline)) {
    if (nxs >= 4) run(std::integral_constant<int, 4>{}, dma_c);
    else if (nxs == 3) run(std::integral_constant<int, 3>{}, dma_c);
    else if (nxs == 2) run(std::integral_constant<int, 2>{}, dma_c);
    else if (nxs == 1) run(std::integral_constant<int, 1>{}, dma_c);
    else run(std::integral_constant<int, 0>{}, dma_c);
  };
  if (wv < 4) by_nxs(std::true_type{});
  else by_nxs(std::false_type{});
  // the empty loads still in flight end before the workgroup does, and before
  // the epilogue writes their LDS
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");

  // lane: output row i0 + 128 iw + 32 qx + l32; register group gr holds columns
  // j0 + 64 jw + 32 qy + 8 gr + 4 half + 0..3
  if (OUT_F32) {
    int64_t dsts[4];      // before any store: a load issued after one waits for it
#pragma unroll
    for (int qx = 0; qx < 4; ++qx) {
      const int64_t i = i0 + iw * 128 + qx * 32 + l32;
      dsts[qx] = i >= i_end ? -1 : (a.row_map ? (int64_t)a.row_map[i] : i);
    }
#pragma unroll
    for (int qx = 0; qx < 4; ++qx) {
      if (dsts[qx] < 0 || dsts[qx] >= a.c_rows) continue;
      float* crow = (float*)a.C + dsts[qx] * a.J;
#pragma unroll
      for (int qy = 0; qy < 2; ++qy) {
#pragma unroll
        for (int gr = 0; gr < 4; ++gr) {
          const int64_t j = j0 + jw * 64 + qy * 32 + 8 * gr + 4 * half;
          const v16f& v = acc[qy][qx];
          if (j < a.J)
            *(float4*)(crow + j) = make_float4(v[4 * gr], v[4 * gr + 1], v[4 * gr + 2], v[4 * gr + 3]);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  } else {
    // through the idle LDS, so that the stores write whole 512-byte row segments
#pragma unroll
    for (int qx = 0; qx < 4; ++qx) {
      const int row = iw * 128 + qx * 32 + l32;
#pragma unroll
      for (int qy = 0; qy < 2; ++qy) {
        const v16f& v = acc[qy][qx];
        // trading groups with lane l ^ 32 leaves each lane 8 consecutive columns
#pragma unroll
        for (int pr = 0; pr < 2; ++pr) {
          const int g0 = 8 * pr, g1 = 8 * pr + 4;
          const auto x = __builtin_amdgcn_permlane32_swap(pack_bf16x2_rne(v[g0], v[g0 + 1]),
                                                          pack_bf16x2_rne(v[g1], v[g1 + 1]), false, false);
          const auto y = __builtin_amdgcn_permlane32_swap(pack_bf16x2_rne(v[g0 + 2], v[g0 + 3]),
                                                          pack_bf16x2_rne(v[g1 + 2], v[g1 + 3]), false, false);
          const int col = jw * 64 + qy * 32 + 16 * pr + 8 * half;
          *(v4i*)(smem + row * kOutPitch + col * 2) = (v4i){(int)x[0], (int)y[0], (int)x[1], (int)y[1]};
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    __syncthreads();
    // 16 bytes (8 columns, wholly inside or past J) of row 16 it + tid / 32; the
    // output is not read here: streaming stores leave the operands in L2
    const int c8 = (tid & 31) * 8;
    const int64_t j = j0 + c8;
    int dst[kBM / 16];
#pragma unroll
    for (int it = 0; it < kBM / 16; ++it) {
      const int64_t i = i0 + it * 16 + (tid >> 5);
      dst[it] = i < i_end ? (a.row_map ? a.row_map[i] : (int)i) : -1;
    }
#pragma unroll 4
    for (int it = 0; it < kBM / 16; ++it) {
      const v4i w = *(const v4i*)(smem + (it * 16 + (tid >> 5)) * kOutPitch + c8 * 2);
      if (dst[it] >= 0 && dst[it] < a.c_rows && j < a.J)
        __builtin_nontemporal_store(w, (v4i*)((uint16_t*)a.C + (int64_t)dst[it] * a.J + j));
    }
  }
}

// Number of groups that can hold rows.
static int64_t live_groups(int64_t I, int64_t E) { return std::min(E, I); }

// Small workgroups that cover the output, from the row count alone: each group
// may add a partial tile.
static int64_t small_count(int64_t I, int64_t J, int64_t E) {
  return (I / kSmBM + live_groups(I, E)) * ((J + kSmBN - 1) / kSmBN);
}

// Small workgroups while there are about 2.5 of them per CU, the large tiles past
// that.  Measured, E4M3 rows, small / large, us:
//   E  1 4096 x 4096:   1 row 7 / 23    256 rows (640) 30 / 38   384 (896) 44 / 38
//   E  2 4096 x 5120:   1 row 8 / 27    64 rows (512) 19 / 31    256 (1280) 68 / 47
//   E  8 2048 x 7168:   1 row 18 / 36   16 rows (640) 24 / 36    64 (1024) 48 / 41
//   E 16 8192 x 5120:   1 row (4096) 124 / 94, 256 rows 1097 / 151
static bool small_tiles(int64_t I, int64_t J, int64_t E) { return small_count(I, J, E) <= 640; }

// Every small workgroup quantizes its own rows where that is less than a launch:
// one workgroup per CU, and up to 65536 values of 16-row tiles each (by the average
// group, as offsets stay on the device: where one of many experts has all rows its
// workgroups quantize up to four times that).  Measured in a graph, quantizer and product / one kernel, us (a call from the host saves 2.5
// more):
//   E 2  512 x  256:  1 row 6.6 / 5.2    64 rows (16384 values) 7.9 / 7.9
//   E 4 1024 x  512:  1 row 6.7 / 5.6    64 rows (32768) 8.5 / 9.7
//   E 1 4096 x 4096:  1 row 8.9 / 7.6    16 rows (65536) 10.7 / 10.3   32 13.1 / 16.4
//   E 8 2048 x 7168:  1 row (114688, two workgroups per CU) 20.8 / 22.5
bool fp4_gemm_takes_bf16(int64_t I, int64_t J, int64_t Kc, int64_t E) {
  if (I == 0 || small_count(I, J, E) > 256) return false;
  const int64_t rows = (I + live_groups(I, E) - 1) / live_groups(I, E);
  return std::min<int64_t>(kSmBM, (rows + 15) / 16 * 16) * Kc <= 65536;
}

template <int XF, bool OUT_F32, bool BF16>
static hipError_t launch_small(const Fp4GemmArgs& a, hipStream_t st) {
  hipLaunchKernelGGL((fp4_rows_small_kernel<XF, OUT_F32, BF16>),
                     dim3((unsigned)rows::grid<kSmBM, kSmBN>(a.I, a.J, a.E)), dim3(kSmWaves * 64), 0, st, a);
  return hipGetLastError();
}

template <int XF, bool OUT_F32>
static hipError_t launch_rows(const Fp4GemmArgs& a, hipStream_t st) {
  if (small_tiles(a.I, a.J, a.E)) return launch_small<XF, OUT_F32, false>(a, st);
  const size_t lds = (size_t)Stage<XF>::kBytes * Stage<XF>::kBufs;
  const hipError_t e = hipFuncSetAttribute((const void*)fp4_rows_kernel<XF, OUT_F32>,
                                           hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((fp4_rows_kernel<XF, OUT_F32>), dim3((unsigned)rows::grid<kBM, kBN>(a.I, a.J, a.E)),
                     dim3(kThreads), lds, st, a);
  return hipGetLastError();
}

hipError_t launch_fp4_gemm(const Fp4GemmArgs& a, hipStream_t st) {
  if (a.I == 0 || a.J == 0) return hipSuccess;
  if (a.A) return a.x_fp4 ? launch_small<kFmtE2M1, false, true>(a, st) : launch_small<kFmtE4M3, false, true>(a, st);
  if (a.x_fp4) return a.out_f32 ? launch_rows<kFmtE2M1, true>(a, st) : launch_rows<kFmtE2M1, false>(a, st);
  return a.out_f32 ? launch_rows<kFmtE4M3, true>(a, st) : launch_rows<kFmtE4M3, false>(a, st);
}

}  // namespace mxk
