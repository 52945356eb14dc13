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
// All are streaming passes, bound by HBM and the vector unit: bytes per h element 4 + 2 (+ 2.06) in
// swiglu_fwd, 2 + 2.06 + 4 in swiglu_bwd, 4 + 4.12 in swiglu_quantize_fwd, 2 +
// 2.06 + 4.12 in swiglu_quantize_bwd.
#include "mx_device.h"
#include "mx_kernels.h"
#include "mx_quantize.h"
#include "mx_swiglu.h"

namespace mxk {

namespace {

constexpr int kThreads = 256;

constexpr uint32_t kFarGate = 0x4280;       // bf16 bits of 64: below, sigmoid_near serves
constexpr uint32_t kFarByte = 124;          // a block of this scale byte holds at most 448 * 2^-3 = 56

// Conversions to E4M3 saturate from here on, to +-448 (bit 23 of the MODE register).  To the
// compiler a conversion has nothing to do with that register: what keeps it behind the change
// is the 0 returned here, whose value the compiler cannot know and which goes into the address
// of what is converted.
__device__ __forceinline__ int saturate_conversions() {
  __builtin_amdgcn_s_setreg(1 | (23 << 6), 1);
  int zero = 0;
  asm volatile("" : "+s"(zero));
  return zero;
}

// Scale bytes need the exponents of the largest magnitudes alone: two at a time, the
// high halves of their fp32 bits packed in a dword.  A half from 0x7F80 on is not finite.
__device__ __forceinline__ uint32_t pack_high(uint32_t lo, uint32_t hi) {
  return __builtin_amdgcn_perm(hi, lo, 0x07060302);
}
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t,
                            __builtin_elementwise_max(__builtin_bit_cast(us2, a), __builtin_bit_cast(us2, b)));
}
__device__ __forceinline__ uint32_t quad_max2(uint32_t v) {
  v = max2(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, false));
  return max2(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, false));
}
__device__ __forceinline__ uint32_t bytes_of(uint32_t highs) {
  const us2 e = __builtin_bit_cast(us2, highs) >> 7;
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(e, (us2){8, 8}) - (us2){8, 8});
}
__device__ __forceinline__ bool not_finite2(uint32_t highs) {
  return max(highs & 0xFFFFu, highs >> 16) >= 0x7F80u;
}
__device__ __forceinline__ bool not_finite(uint32_t high) { return high >= 0x7F80u; }

// A byte's scale as the conversions take it: the float whose exponent field it is.
__device__ __forceinline__ float scale_bits(uint32_t byte) { return __uint_as_float(byte << 23); }

__device__ __forceinline__ uint32_t absmax(const float* x, int n, int step) {
  float m = __builtin_fabsf(x[0]);
#pragma unroll
  for (int i = 1; i < n; ++i) m = __builtin_elementwise_maximum(m, __builtin_fabsf(x[i * step]));   // a NaN stays one
  return __float_as_uint(m);
}

// Four values -> codes, saturating (see saturate_conversions).
__device__ __forceinline__ int codes4(float a, float b, float c, float d, float scale) {
  s16x2 r = {0, 0};
  r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, a, b, scale, 0);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, c, d, scale, 1);
  return __builtin_bit_cast(int, r);
}
__device__ __forceinline__ v2i codes8(const float* x, uint32_t byte) {
  const float scale = scale_bits(byte);
  return (v2i){codes4(x[0], x[1], x[2], x[3], scale), codes4(x[4], x[5], x[6], x[7], scale)};
}
__device__ __forceinline__ v2i codes8(v4i x, uint32_t byte) {
  const float scale = scale_bits(byte);
  v2i q;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    s16x2 r = {0, 0};
    r = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(r, __builtin_bit_cast(bf16x2_t, (uint32_t)x[2 * i]), scale, 0);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(r, __builtin_bit_cast(bf16x2_t, (uint32_t)x[2 * i + 1]), scale, 1);
    q[i] = __builtin_bit_cast(int, r);
  }
  return q;
}

// Codes of eight values each of two blocks spread over a quad, whose largest
// magnitudes' high halves are `highs`; their bytes, the second in bits 16 to 23.
template <class X>
__device__ __forceinline__ uint32_t quantize2(const X& x, const X& y, uint32_t highs, v2i& qx, v2i& qy) {
  uint32_t bytes = bytes_of(highs);
  qx = codes8(x, bytes & 0xFFu);
  qy = codes8(y, bytes >> 16);
  if (__any(not_finite2(highs))) {
    const v2i nan = {0x7F7F7F7F, 0x7F7F7F7F};
    const bool bx = not_finite(highs & 0xFFFFu), by = not_finite(highs >> 16);
    qx = bx ? nan : qx;
    qy = by ? nan : qy;
    bytes = (bx ? 0xFFu : bytes & 0xFFu) | (by ? 0xFF0000u : bytes & 0xFF0000u);
  }
  return bytes;
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

// Eight codes -> their values (of a block of byte 255, which holds NaN, anything).
__device__ __forceinline__ void finite8(v2i codes, uint32_t byte, float* out) {
  const float scale = scale_bits(byte);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const v2f a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8((uint32_t)codes[i], scale, false);
    const v2f b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8((uint32_t)codes[i], scale, true);
    out[4 * i] = a[0];
    out[4 * i + 1] = a[1];
    out[4 * i + 2] = b[0];
    out[4 * i + 3] = b[1];
  }
}

}  // namespace

// One thread per eight columns of h.  A DPP quad holds a block of 32.  The vector unit
// has as much to do as HBM: the whole-range sigmoid, whose far branch a wave takes only
// where one of its gates is beyond 64 (the same result for the others), conversions
// that saturate by themselves and streamed stores took 16384 x 8192 forward from 217
// to 172 us and backward from 212 to 171 us (6.3 TB/s; 1.08 GB each); 4099 x 2048 takes
// 15 us each.
template <bool KEEP>
__global__ __launch_bounds__(kThreads) void swiglu_fwd_kernel(const uint16_t* __restrict__ gu, int64_t chunks,
                                                              int64_t N, uint16_t* __restrict__ h,
                                                              uint8_t* __restrict__ kept, uint8_t* __restrict__ kept_s) {
  const int64_t i = wide_block() * kThreads + threadIdx.x;
  if (i >= chunks) return;
  const int zero = saturate_conversions();
  int64_t row, c;
  row_of(i, N / 8, row, c);
  const uint16_t* src = gu + zero + row * 2 * N + 8 * c;
  const v4i gw = __builtin_nontemporal_load((const v4i*)src);
  const v4i uw = __builtin_nontemporal_load((const v4i*)(src + N));
  float g[8], u[8], o[8];
  floats8(gw, g);
  floats8(uw, u);
  const us2 mg = absmax8x2(gw), mu = absmax8x2(uw);
  uint32_t highs = max((uint32_t)mg[0], (uint32_t)mg[1]) | max((uint32_t)mu[0], (uint32_t)mu[1]) << 16;
  if (__any((highs & 0xFFFFu) >= kFarGate)) {
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = silu_mul(g[j], u[j]);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = g[j] * sigmoid_near(g[j]).m * u[j];
  }
  __builtin_nontemporal_store(pack8(o), (v4i*)(h + row * N + 8 * c));
  if (KEEP) {
    v2i gq, uq;
    const uint32_t bytes = quantize2(gw, uw, quad_max2(highs), gq, uq);
    uint8_t* dst = kept + row * 2 * N + 8 * c;
    __builtin_nontemporal_store(gq, (v2i*)dst);
    __builtin_nontemporal_store(uq, (v2i*)(dst + N));
    if ((c & 3) == 0) {
      uint8_t* s = kept_s + row * (N / 16) + (c >> 2);
      s[0] = (uint8_t)bytes;
      s[N / 32] = (uint8_t)(bytes >> 16);
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
  const uint32_t gb = s[0], ub = s[N / 32];
  finite8(gq, gb, g);
  finite8(uq, ub, u);
  if (__any(gb > kFarByte || ub == 0xFFu)) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float x = gb == 0xFFu ? __builtin_nanf("") : g[j], y = ub == 0xFFu ? __builtin_nanf("") : u[j];
      const Sigmoid p = sigmoid_parts(x);
      dg[j] = scaled(p, p.m * fmaf(x, p.q, 1.f), d[j] * y);
      du[j] = scaled(p, x * p.m, d[j]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const Sigmoid p = sigmoid_near(g[j]);
      dg[j] = p.m * fmaf(g[j], p.q, 1.f) * (d[j] * u[j]);
      du[j] = g[j] * p.m * d[j];
    }
  }
  uint16_t* dst = dgu + row * 2 * N + 8 * c;
  __builtin_nontemporal_store(pack8(dg), (v4i*)dst);
  __builtin_nontemporal_store(pack8(du), (v4i*)(dst + N));
}

// ---------------------------------------------------------------------------
// Between two products of routed experts.  A workgroup of eight waves takes 128
// rows and 128 columns of h; wave w rows 32 (w/2).., one block of the colwise
// quantization, and columns 64 (w%2)..; lane l rows 4 (l/8) + i (i < 4) and eight
// columns 8 (l%8)..: a quad holds a block of 32 columns, the lanes l%8 + 8j one of 32
// rows.  Codes of the rows go straight out; those of the columns through LDS, and
// out as whole lines.  Row r belongs to item rows[r]; a row with none (padding,
// behind the last group) holds anything and counts as zeros.
//
// 4 rows a lane instead of 8 hold both of the backward's gradients in fp32 in 128
// registers, so that two workgroups share a CU and one computes while the other
// waits for memory.  16896 x 8192 (0.14 G of h): forward 197 us (5.6 TB/s; 327 with 8 rows a
// lane and conversions in steps), inference 117 us (5.8), backward 264 us (4.3; 447), where
// plain vector instructions fill three issue slots in five and reciprocals, powers and
// conversions take several each; its waves wait for memory or LDS in 42% of their cycles, for
// a slot in 33%.  Over two sets of tensors in turn: 226, 125 and 226 us.
// ---------------------------------------------------------------------------
namespace {

constexpr int kTileRows = 128, kTileCols = 128, kTileThreads = 512, kLaneRows = 4;

struct Place {
  int cp, rg, wr, wc, row, col;             // row and col: of the lane's first value within the tile
  __device__ __forceinline__ Place() {
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    cp = lane & 7;
    rg = lane >> 3;
    wr = wv >> 1;
    wc = wv & 1;
    row = 32 * wr + kLaneRows * rg;
    col = 64 * wc + 8 * cp;
  }
};

struct ColCodes {
  uint8_t codes[kTileCols * kTileRows];     // [column][row], see code_at
  uint8_t scales[4 * kTileCols];            // [block][column]
};

// Where 16-byte slot s (16 rows) of a column lies.  Neighbouring groups of eight
// columns take the halves of a 256-byte line in opposite order, and every second one
// another slot: a wave's writes (eight groups x eight lanes of 4 bytes) and reads (eight slots
// of eight columns) are spread evenly over 64 banks.  The writes are not free of conflicts for
// that: half a wave goes at a time, over 32 banks, where the two halves of a line coincide, and
// each write takes four cycles, two of them counted as conflicts (most of the kernels'
// count).  They are hidden: without these writes the kernels take as long.
__device__ __forceinline__ int code_at(int col, int s) {
  return (col ^ (col >> 3 & 1)) * kTileRows + 16 * (s ^ (2 * (col >> 4 & 3)));
}

// Byte b of `x` into byte i of `bytes`.
__device__ __forceinline__ uint32_t put_byte(uint32_t bytes, int i, uint32_t x) { return bytes | x << (8 * i); }

// Colwise codes of the lane's 4 rows x 8 columns into LDS.
__device__ __forceinline__ void put_columns(ColCodes& lds, const float (&x)[kLaneRows][8], const Place& p) {
  uint32_t scales[2] = {0, 0};
#pragma unroll
  for (int c = 0; c < 8; c += 2) {
    uint32_t m = pack_high(absmax(&x[0][c], kLaneRows, 8), absmax(&x[0][c + 1], kLaneRows, 8));
    m = max2(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x128, 0xF, 0xF, false));    // lanes 8 apart (row_ror:8)
    const auto a = __builtin_amdgcn_permlane16_swap(m, m, false, false);                 // 16
    m = max2(a[0], a[1]);
    const auto b = __builtin_amdgcn_permlane32_swap(m, m, false, false);                 // 32
    m = max2(b[0], b[1]);
    uint32_t bytes = bytes_of(m);
    int q[2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
      q[h] = codes4(x[0][c + h], x[1][c + h], x[2][c + h], x[3][c + h], scale_bits(h ? bytes >> 16 : bytes & 0xFFu));
    if (__any(not_finite2(m))) {
      const bool b0 = not_finite(m & 0xFFFFu), b1 = not_finite(m >> 16);
      q[0] = b0 ? 0x7F7F7F7F : q[0];
      q[1] = b1 ? 0x7F7F7F7F : q[1];
      bytes = (b0 ? 0xFFu : bytes & 0xFFu) | (b1 ? 0xFF0000u : bytes & 0xFF0000u);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) *(int*)(lds.codes + code_at(p.col + c + h, p.row >> 4) + (p.row & 15)) = q[h];
    scales[c >> 2] |= ((bytes | bytes >> 8) & 0xFFFFu) << (8 * (c & 2));
  }
  if (p.rg == 0) *(v2i*)(lds.scales + kTileCols * p.wr + p.col) = (v2i){(int)scales[0], (int)scales[1]};
}

// Four bytes `stride` apart as a dword: the four blocks of a row or column.
__device__ __forceinline__ uint32_t gather4(const uint8_t* p, int stride) {
  return (uint32_t)p[0] | (uint32_t)p[stride] << 8 | (uint32_t)p[2 * stride] << 16 | (uint32_t)p[3 * stride] << 24;
}

// ... and from there to columns k0.. of q_t [., ldq] and s_t [ldq/128][cols][4].
__device__ __forceinline__ void store_columns(const ColCodes& lds, int64_t n0, int64_t k0, int64_t cols, int64_t ldq,
                                              uint8_t* __restrict__ q_t, uint8_t* __restrict__ s_t) {
  const int tid = threadIdx.x, s = tid & 7;
#pragma unroll
  for (int it = 0; it < kTileCols * 8 / kTileThreads; ++it) {
    const int k = (tid >> 3) + kTileThreads / 8 * it;
    __builtin_nontemporal_store(*(const v4i*)(lds.codes + code_at(k, s)), (v4i*)(q_t + (k0 + k) * ldq + n0 + 16 * s));
  }
  if (tid < kTileCols) *(uint32_t*)(s_t + (n0 >> 7) * cols * 4 + (k0 + tid) * 4) = gather4(lds.scales + tid, kTileCols);
}

// Tile of a workgroup of the backward.  Workgroups go round the 8 XCDs: of every
// eight rows of tiles each XCD takes one, whose lines its own L2 then reads and writes
// in their order (16384 x 8192: 262 us for 279).  The forward, which reads whole lines
// of 256 bytes, gains nothing (226 us in the grid's order, 236 so).
struct Tile {
  uint32_t x, y;
  __device__ __forceinline__ Tile() {
    const uint32_t nx = gridDim.x, b = blockIdx.y * nx + blockIdx.x, eight = b / (8 * nx), in = b % (8 * nx);
    const bool whole = eight < gridDim.y / 8;
    x = whole ? in >> 3 : blockIdx.x;
    y = whole ? 8 * eight + (in & 7) : blockIdx.y;
  }
};

// Item of row r, or -1.
__device__ __forceinline__ int item_of(const SwigluArgs& a, int64_t r) {
  if (r >= a.M) return -1;
  const int64_t item = a.rows ? (int64_t)a.rows[r] : r;
  return item >= 0 && item < a.n_items ? (int)item : -1;
}

}  // namespace

template <bool TRAIN>
__global__ __launch_bounds__(kTileThreads) __attribute__((amdgpu_waves_per_eu(4))) void swiglu_quantize_fwd_kernel(
    SwigluArgs a) {
  __shared__ __attribute__((aligned(16))) ColCodes lds;
  __shared__ __attribute__((aligned(16))) uint8_t srow[3][4 * kTileRows];      // [block][row] of h, gate, up
  const Place p;
  const int tid = threadIdx.x, blk = 2 * p.wc + (p.cp >> 2);
  const int64_t n0 = (int64_t)blockIdx.y * kTileRows, k0 = (int64_t)blockIdx.x * kTileCols;
  const int64_t r0 = n0 + p.row, c0 = k0 + p.col;
  const int zero = saturate_conversions();
  int item[kLaneRows];
#pragma unroll
  for (int i = 0; i < kLaneRows; ++i) item[i] = item_of(a, r0 + i);
  v4i gw[kLaneRows], uw[kLaneRows];
#pragma unroll
  for (int i = 0; i < kLaneRows; ++i) {
    gw[i] = uw[i] = (v4i){0, 0, 0, 0};
    if (item[i] >= 0) {
      const uint16_t* src = a.gu + zero + (r0 + i) * 2 * a.N + c0;
      gw[i] = __builtin_nontemporal_load((const v4i*)src);
      uw[i] = __builtin_nontemporal_load((const v4i*)(src + a.N));
    }
  }
  float w[kLaneRows];
#pragma unroll
  for (int i = 0; i < kLaneRows && TRAIN; ++i) w[i] = item[i] < 0 ? 0.f : a.combine ? a.combine[item[i]] : 1.f;
  float h[kLaneRows][8];
  uint32_t sh = 0, sg = 0, su = 0;                // the rows' scale bytes
#pragma unroll
  for (int i = 0; i < kLaneRows; ++i) {
    const int64_t r = r0 + i;
    float g[8], u[8];
    floats8(gw[i], g);
    floats8(uw[i], u);
    // largest magnitudes of the gate and up values, packed
    const us2 mg = absmax8x2(gw[i]), mu = absmax8x2(uw[i]);
    uint32_t highs = max((uint32_t)mg[0], (uint32_t)mg[1]) | max((uint32_t)mu[0], (uint32_t)mu[1]) << 16;
    if (TRAIN) {
      highs = quad_max2(highs);
      v2i gq, uq;
      const uint32_t bytes = quantize2(gw[i], uw[i], highs, gq, uq);
      if (r < a.M) {
        uint8_t* dst = a.kept + r * 2 * a.N + c0;
        *(v2i*)dst = gq;
        *(v2i*)(dst + a.N) = uq;
      }
      sg = put_byte(sg, i, bytes & 0xFFu);
      su = put_byte(su, i, bytes >> 16);
    }
    if (__any((highs & 0xFFFFu) >= kFarGate)) {
#pragma unroll
      for (int c = 0; c < 8; ++c) h[i][c] = silu_mul(g[c], u[c]);
    } else {
#pragma unroll
      for (int c = 0; c < 8; ++c) h[i][c] = g[c] * sigmoid_near(g[c]).m * u[c];
    }
  }
  // two rows of h at a time
#pragma unroll
  for (int i = 0; i < kLaneRows; i += 2) {
    v2i q0, q1;
    const uint32_t bytes = quantize2(h[i], h[i + 1], quad_max2(pack_high(absmax(h[i], 8, 1), absmax(h[i + 1], 8, 1))),
                                     q0, q1);
    if (r0 + i < a.M) *(v2i*)(a.q + (r0 + i) * a.N + c0) = q0;
    if (r0 + i + 1 < a.M) *(v2i*)(a.q + (r0 + i + 1) * a.N + c0) = q1;
    sh = put_byte(put_byte(sh, i, bytes & 0xFFu), i + 1, bytes >> 16);
  }
  if ((p.cp & 3) == 0) {
    *(uint32_t*)(srow[0] + blk * kTileRows + p.row) = sh;
    if (TRAIN) {
      *(uint32_t*)(srow[1] + blk * kTileRows + p.row) = sg;
      *(uint32_t*)(srow[2] + blk * kTileRows + p.row) = su;
    }
  }
#pragma unroll
  for (int i = 0; i < kLaneRows && TRAIN; ++i)
#pragma unroll
    for (int c = 0; c < 8; ++c) h[i][c] *= w[i];
  if (TRAIN) put_columns(lds, h, p);
  __syncthreads();
  {
    const int part = tid / kTileRows, r = tid % kTileRows;      // scales of h, of the gate and of the up values
    if (part < (TRAIN ? 3 : 1) && n0 + r < a.M) {
      uint8_t* s = part == 0 ? a.s : a.kept_s + (part == 2 ? a.N >> 7 : 0) * a.M * 4;
      *(uint32_t*)(s + (k0 >> 7) * a.M * 4 + (n0 + r) * 4) = gather4(srow[part] + r, kTileRows);
    }
  }
  if (TRAIN) store_columns(lds, n0, k0, a.N, a.ldq, a.q_t, a.s_t);
}

__global__ __launch_bounds__(kTileThreads) __attribute__((amdgpu_waves_per_eu(4))) void swiglu_quantize_bwd_kernel(
    SwigluArgs a) {
  __shared__ __attribute__((aligned(16))) ColCodes lds[2];
  __shared__ __attribute__((aligned(16))) uint8_t srow[2][4 * kTileRows];      // [block][row] of dg, du
  __shared__ float dots[2][kTileRows];
  const Place p;
  const int tid = threadIdx.x, blk = 2 * p.wc + (p.cp >> 2);
  const Tile tile;
  const int64_t n0 = (int64_t)tile.y * kTileRows, k0 = (int64_t)tile.x * kTileCols;
  const int64_t r0 = n0 + p.row, c0 = k0 + p.col;
  const int zero = saturate_conversions();
  int item[kLaneRows];
#pragma unroll
  for (int i = 0; i < kLaneRows; ++i) item[i] = item_of(a, r0 + i);
  v4i dw[kLaneRows];
  v2i gq[kLaneRows], uq[kLaneRows];
  uint32_t gs[kLaneRows], us[kLaneRows];
#pragma unroll
  for (int i = 0; i < kLaneRows; ++i) {
    const int64_t r = r0 + i;
    dw[i] = (v4i){0, 0, 0, 0};
    gq[i] = uq[i] = (v2i){0, 0};
    gs[i] = us[i] = 0;
    if (item[i] >= 0) {
      // (streaming loads: 262 us instead of 245)
      dw[i] = *(const v4i*)(a.dh + zero + r * a.N + c0);
      const uint8_t* src = a.kept + r * 2 * a.N + c0;
      gq[i] = *(const v2i*)src;
      uq[i] = *(const v2i*)(src + a.N);
      const uint8_t* s = a.kept_s + (k0 >> 7) * a.M * 4 + r * 4;
      gs[i] = *(const uint32_t*)s;
      us[i] = *(const uint32_t*)(s + (a.N >> 7) * a.M * 4);
    }
  }
  float w[kLaneRows];
#pragma unroll
  for (int i = 0; i < kLaneRows; ++i) w[i] = item[i] < 0 ? 0.f : a.combine ? a.combine[item[i]] : 1.f;
  float dg[kLaneRows][8], du[kLaneRows][8];
  uint32_t sg = 0, su = 0;                        // the rows' scale bytes
#pragma unroll
  for (int i = 0; i < kLaneRows; ++i) {
    const int64_t r = r0 + i;
    const uint32_t gb = gs[i] >> (8 * blk) & 0xFFu, ub = us[i] >> (8 * blk) & 0xFFu;
    float d[8], g[8], u[8];
    floats8(dw[i], d);
    finite8(gq[i], gb, g);
    finite8(uq[i], ub, u);
    float dot = 0.f;
    if (__any(gb > kFarByte || ub == 0xFFu)) {
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const float x = gb == 0xFFu ? __builtin_nanf("") : g[c], y = ub == 0xFFu ? __builtin_nanf("") : u[c];
        const Sigmoid s = sigmoid_parts(x);
        const float e = w[i] * d[c], xs = x * s.m;
        dg[i][c] = scaled(s, s.m * fmaf(x, s.q, 1.f), e * y);
        du[i][c] = scaled(s, xs, e);
        dot = fmaf(d[c], scaled(s, xs, y), dot);
      }
    } else {
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const Sigmoid s = sigmoid_near(g[c]);
        const float e = w[i] * d[c], xs = g[c] * s.m;
        dg[i][c] = s.m * fmaf(g[c], s.q, 1.f) * (e * u[c]);
        du[i][c] = xs * e;
        dot = fmaf(d[c], xs * u[c], dot);
      }
    }
    if (a.partial) {
      // over the eight lanes of a row
      dot += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(dot), 0x141, 0xF, 0xF, false));   // half mirror
      dot += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(dot), 0x4E, 0xF, 0xF, false));    // quad [2,3,0,1]
      dot += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(dot), 0xB1, 0xF, 0xF, false));    // quad [1,0,3,2]
      if (p.cp == 0) dots[p.wc][p.row + i] = dot;
    }
    v2i qg, qu;
    const uint32_t bytes =
        quantize2(dg[i], du[i], quad_max2(pack_high(absmax(dg[i], 8, 1), absmax(du[i], 8, 1))), qg, qu);
    if (r < a.M) {
      uint8_t* dst = a.q + r * 2 * a.N + c0;
      *(v2i*)dst = qg;
      *(v2i*)(dst + a.N) = qu;
    }
    sg = put_byte(sg, i, bytes & 0xFFu);
    su = put_byte(su, i, bytes >> 16);
  }
  if ((p.cp & 3) == 0) {
    *(uint32_t*)(srow[0] + blk * kTileRows + p.row) = sg;
    *(uint32_t*)(srow[1] + blk * kTileRows + p.row) = su;
  }
  put_columns(lds[0], dg, p);
  put_columns(lds[1], du, p);
  __syncthreads();
  {
    const int part = tid / kTileRows, r = tid % kTileRows;      // scales of dg and of du, sums of the rows
    if (part < 2 && n0 + r < a.M)
      *(uint32_t*)(a.s + ((part * a.N + k0) >> 7) * a.M * 4 + (n0 + r) * 4) = gather4(srow[part] + r, kTileRows);
    if (part == 2 && a.partial && n0 + r < a.M) a.partial[(int64_t)tile.x * a.M + n0 + r] = dots[0][r] + dots[1][r];
  }
  store_columns(lds[0], n0, k0, 2 * a.N, a.ldq, a.q_t, a.s_t);
  store_columns(lds[1], n0, a.N + k0, 2 * a.N, a.ldq, a.q_t, a.s_t);
}

// dcombine[rows[r]] = sum over the column tiles of row r, in a fixed order, where pos
// agrees; items without such a row get 0.  64 rows per workgroup, every fourth tile per
// wave; 5 us for 33792 rows.
__global__ __launch_bounds__(kThreads) void swiglu_dcombine_kernel(SwigluArgs a, float* __restrict__ dcombine) {
  __shared__ float part[kThreads];
  const int wv = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t r = wide_block() * 64 + lane;
  const int64_t tiles = a.N / kTileCols;
  float sum = 0.f;
  if (r < a.M) {
#pragma unroll 8
    for (int64_t t = wv; t < tiles; t += 4) sum += a.partial[t * a.M + r];
  }
  part[threadIdx.x] = sum;
  __syncthreads();
  if (wv != 0) return;
  // every item is written once, whatever rows and pos hold: by its row where the two agree, else here
  if (r < a.n_items && a.pos) {
    const int64_t row = a.pos[r];
    if (row < 0 || row >= a.M || a.rows[row] != r) dcombine[r] = 0.f;
  }
  const int item = item_of(a, r);
  if (item >= 0 && (!a.pos || a.pos[item] == r))
    dcombine[item] = part[lane] + part[64 + lane] + part[128 + lane] + part[192 + lane];
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
  hipLaunchKernelGGL(swiglu_dcombine_kernel, wide_grid((n + 63) / 64), dim3(kThreads), 0, st, a, dcombine);
  return hipGetLastError();
}

}  // namespace mxk
