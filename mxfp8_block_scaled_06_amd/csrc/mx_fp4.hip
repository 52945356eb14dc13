// MXFP4 quantizers and dequantizer for gfx950.
//
// MXFP4 is the 4-bit sibling of the library's MXFP8: 32 values along the
// contraction share one E8M0 byte, byte = clamp(floor(log2 amax) - 2, -127,
// 127) + 127 (2 is E2M1's largest exponent), and every element is
// value * 2^(127 - byte) rounded to nearest even on the E2M1 grid
// {0, 0.5, 1, 1.5, 2, 3, 4, 6}, saturated to +-6, sign kept on zeros.  An
// all-zero block has byte 0; a block that holds NaN or Inf has byte 0xFF and
// zero codes (E2M1 has no NaN; the scale byte alone makes the block's products
// NaN in the matrix cores).  Two codes to a byte, the even element of the
// contraction axis in the low four bits.
//
// All of it is HBM-bound streaming (65600 x 5120: quantized in 140 us, 6.1 TB/s,
// restored in 151, 5.6 TB/s; the weights of 16 x 8192 x 5120 in both orientations
// in 356 us, 5.8 TB/s, restored from one in 300 to 340): the amax is an integer
// max over |bf16| bits, the scale its exponent field, and
// v_cvt_scalef32_pk_fp4_bf16 scales, rounds to nearest even and saturates two
// values in one instruction.
#include "mx_device.h"
#include "mx_kernels.h"
#include "mx_quantize.h"

namespace mxk {

constexpr int kF4Threads = 256;

// Two ways over the values, 8 of them (a chunk) per lane and step, a DPP quad on
// one block.  Row-major scales: chunks in order, scale of chunk c at c / 4.  GEMM
// scales [batch][cols/128][rows][4]: tiles of 256 columns (whole 128-byte lines
// of codes) x 8 NC rows, so that a tile's scales are two runs of 4 bytes per
// row; with the chunks in order every lane computed its scale's place with two
// 64-bit divisions and a wave's 16 scales lay in four far lines.
constexpr int kT4Cols = 256, kT4Rows = kF4Threads / 32;   // rows of one step
// Steps per workgroup: 8 keep enough loads in flight for the bandwidth, 1 spreads
// an input of fewer than 1024 such tiles over the CUs.  Restoring 16 x 8192 x 5120:
// 8 steps 338 us, 4 352, 2 372; 4 x 1024 x 512 (128 tiles): 1 step 4.3, 8 steps 7.5
// (quantizing it 3.7 and 4.3 to 5.2).
constexpr int kT4Steps = 8;

inline int t4_steps(int64_t batch, int64_t rows, int64_t cols) {
  return batch * ((rows + kT4Rows * kT4Steps - 1) / (kT4Rows * kT4Steps)) * ((cols + kT4Cols - 1) / kT4Cols) >= 1024
             ? kT4Steps
             : 1;
}

inline dim3 t4_grid(int64_t batch, int64_t rows, int64_t cols, int steps) {
  return wide_grid(batch * ((rows + kT4Rows * steps - 1) / (kT4Rows * steps)) * ((cols + kT4Cols - 1) / kT4Cols));
}

// A workgroup's tile: batch entry, first row and first column, column tiles
// fastest.
struct Tile4 {
  int64_t b, r0;
  int k0;
};
template <int NC>
__device__ __forceinline__ Tile4 tile4(int64_t rows, int cols) {
  const uint32_t kt = (uint32_t)(cols + kT4Cols - 1) / kT4Cols;
  const uint32_t rt = (uint32_t)((rows + kT4Rows * NC - 1) / (kT4Rows * NC));
  const uint32_t id = (uint32_t)wide_block(), t = id / kt;      // at most 2^32 / 4 tiles of a block or more
  Tile4 o;
  o.k0 = (int)(id - t * kt) * kT4Cols;
  o.b = t / rt;
  o.r0 = (int64_t)(t - (uint32_t)o.b * rt) * (kT4Rows * NC);
  return o;
}

// ---------------------------------------------------------------------------
// Rowwise quantizer.
// ---------------------------------------------------------------------------
__global__ __launch_bounds__(kF4Threads) void quant_rowwise_fp4_kernel(const uint16_t* __restrict__ x,
                                                                       int64_t nchunks, uint8_t* __restrict__ q,
                                                                       uint8_t* __restrict__ s) {
  const int64_t idx = wide_block() * kF4Threads + threadIdx.x;
  v4i w = (v4i){0, 0, 0, 0};
  if (idx < nchunks) w = __builtin_nontemporal_load((const v4i*)(x + idx * 8));
  // nchunks is a multiple of 4: a quad is wholly in range or wholly out
  const uint32_t byte = e8m0_fp4_from_absbits(quad_max(absmax8(w)));
  if (idx < nchunks) {
    *(uint32_t*)(q + idx * 4) = quant8_fp4(w, byte);
    if ((threadIdx.x & 3) == 0) s[idx >> 2] = (uint8_t)byte;
  }
}

template <int NC>
__global__ __launch_bounds__(kF4Threads) void quant_tiles_fp4_kernel(const uint16_t* __restrict__ x, int64_t batch,
                                                                     int64_t rows, int cols, uint8_t* __restrict__ q,
                                                                     uint8_t* __restrict__ s) {
  __shared__ uint8_t sc[2][kT4Rows * NC][4];     // [chunk of 128][row][block]
  const Tile4 t = tile4<NC>(rows, cols);
  if (t.b >= batch) return;
  const int pc = threadIdx.x & 31, r = threadIdx.x >> 5;
  const bool k_in = t.k0 + 8 * pc < cols;
  v4i w[NC];
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int64_t row = t.r0 + kT4Rows * i + r;
    w[i] = (v4i){0, 0, 0, 0};
    if (k_in && row < rows)
      w[i] = __builtin_nontemporal_load((const v4i*)(x + (t.b * rows + row) * cols + t.k0 + 8 * pc));
  }
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int64_t row = t.r0 + kT4Rows * i + r;
    const uint32_t byte = e8m0_fp4_from_absbits(quad_max(absmax8(w[i])));
    if (k_in && row < rows) *(uint32_t*)(q + ((t.b * rows + row) * cols + t.k0) / 2 + 4 * pc) = quant8_fp4(w[i], byte);
    if ((pc & 3) == 0) sc[pc >> 4][kT4Rows * i + r][(pc >> 2) & 3] = (uint8_t)byte;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * kT4Rows * NC; i += kF4Threads) {
    const int ch = i / (kT4Rows * NC), rr = i % (kT4Rows * NC);
    if (t.k0 + 128 * ch < cols && t.r0 + rr < rows)
      *(uint32_t*)(s + (t.b * (cols / 128) + t.k0 / 128 + ch) * rows * 4 + (t.r0 + rr) * 4) =
          *(const uint32_t*)sc[ch][rr];
  }
}

hipError_t launch_quant_rowwise_fp4(const uint16_t* x, int64_t rows_total, int64_t cols, uint8_t* q, uint8_t* s,
                                    int64_t gemm_rows_per_batch, hipStream_t st) {
  const int64_t nchunks = rows_total * (cols / 8);
  if (nchunks == 0) return hipSuccess;
  if (gemm_rows_per_batch == 0) {
    hipLaunchKernelGGL(quant_rowwise_fp4_kernel, wide_grid((nchunks + kF4Threads - 1) / kF4Threads),
                       dim3(kF4Threads), 0, st, x, nchunks, q, s);
    return hipGetLastError();
  }
  const int64_t rows = gemm_rows_per_batch, batch = rows_total / rows;
  const int steps = t4_steps(batch, rows, cols);
  const dim3 grid = t4_grid(batch, rows, cols, steps);
  if (steps == kT4Steps)
    hipLaunchKernelGGL(quant_tiles_fp4_kernel<kT4Steps>, grid, dim3(kF4Threads), 0, st, x, batch, rows, (int)cols,
                       q, s);
  else
    hipLaunchKernelGGL(quant_tiles_fp4_kernel<1>, grid, dim3(kF4Threads), 0, st, x, batch, rows, (int)cols,
                       q, s);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Dequantizer: 8 codes (a dword) per lane -> 8 bf16 values.  Every product
// code * 2^(byte - 127) is a bf16 number (subnormal for the lowest bytes)
// except 4 and 6 at byte 254, which give Inf; byte 0xFF gives NaN.
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t dequant2_bits(uint32_t codes, uint32_t byte) {
  // |code| as a bf16 bit pattern at byte 127: E2M1's 2-bit exponent and
  // 1-bit mantissa become bf16's by a shift, 0.5 (the subnormal) aside
  uint32_t out = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t c = (codes >> (4 * i)) & 15u, m = c & 7u;
    const float v = m == 1u ? 0.5f : __uint_as_float(m == 0u ? 0u : (126u + (m >> 1)) << 23 | (m & 1u) << 22);
    // two exact steps: 2^(byte - 127) itself is subnormal for byte 0
    const float half = byte == 0u ? 0.5f : 1.0f;
    const float p = v * half * __uint_as_float((byte == 0u ? 1u : byte) << 23);
    const uint32_t bits = byte == 0xFFu ? 0x7FC0u : __float_as_uint(p) >> 16;
    out |= (bits | (byte == 0xFFu ? 0u : (c & 8u) << 12)) << (16 * i);
  }
  return out;
}

__device__ __forceinline__ v4i dequant8(uint32_t codes, uint32_t byte) {
  v4i o;
#pragma unroll
  for (int d = 0; d < 4; ++d) o[d] = (int)dequant2_bits(codes >> (8 * d), byte);
  return o;
}

// Chunks per thread, 256 apart: a workgroup writes 16 KB in one piece, and its
// reads are under way before the first store (16 x 8192 x 5120: 283 us, with one
// chunk per thread 390).  One for inputs that would leave CUs idle (4 MB: 3.7 us,
// with four 4.6).
constexpr int kDqChunks = 4;

template <int NC>
__global__ __launch_bounds__(kF4Threads) void dequant_fp4_kernel(const uint8_t* __restrict__ q,
                                                                 const uint8_t* __restrict__ s, int64_t nchunks,
                                                                 uint16_t* __restrict__ out) {
  const int64_t base = wide_block() * (kF4Threads * NC) + threadIdx.x;
  uint32_t c[NC], byte[NC];
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int64_t idx = min(base + i * kF4Threads, nchunks - 1);
    c[i] = *(const uint32_t*)(q + idx * 4);
    byte[i] = s[idx >> 2];
  }
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int64_t idx = base + i * kF4Threads;
    if (idx < nchunks) __builtin_nontemporal_store(dequant8(c[i], byte[i]), (v4i*)(out + idx * 8));
  }
}

template <int NC>
__global__ __launch_bounds__(kF4Threads) void dequant_tiles_fp4_kernel(const uint8_t* __restrict__ q,
                                                                       const uint8_t* __restrict__ s, int64_t batch,
                                                                       int64_t rows, int cols,
                                                                       uint16_t* __restrict__ out) {
  const Tile4 t = tile4<NC>(rows, cols);
  if (t.b >= batch) return;
  const int pc = threadIdx.x & 31, r = threadIdx.x >> 5;
  if (t.k0 + 8 * pc >= cols) return;
  const uint8_t* sb = s + (t.b * (cols / 128) + t.k0 / 128 + (pc >> 4)) * rows * 4 + ((pc >> 2) & 3);
  uint32_t c[NC], byte[NC];
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int64_t row = t.r0 + kT4Rows * i + r;
    c[i] = byte[i] = 0;
    if (row < rows) {
      c[i] = *(const uint32_t*)(q + ((t.b * rows + row) * cols + t.k0) / 2 + 4 * pc);
      byte[i] = sb[row * 4];
    }
  }
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int64_t row = t.r0 + kT4Rows * i + r;
    if (row < rows)
      __builtin_nontemporal_store(dequant8(c[i], byte[i]), (v4i*)(out + (t.b * rows + row) * cols + t.k0 + 8 * pc));
  }
}

hipError_t launch_dequant_fp4(const uint8_t* q, const uint8_t* s, int64_t rows_total, int64_t cols, uint16_t* out,
                              int64_t gemm_rows_per_batch, hipStream_t st) {
  const int64_t nchunks = rows_total * (cols / 8);
  if (nchunks == 0) return hipSuccess;
  if (gemm_rows_per_batch == 0) {
    if (nchunks >= 1024 * kF4Threads * kDqChunks)
      hipLaunchKernelGGL(dequant_fp4_kernel<kDqChunks>,
                         wide_grid((nchunks + kF4Threads * kDqChunks - 1) / (kF4Threads * kDqChunks)),
                         dim3(kF4Threads), 0, st, q, s, nchunks, out);
    else
      hipLaunchKernelGGL(dequant_fp4_kernel<1>, wide_grid((nchunks + kF4Threads - 1) / kF4Threads), dim3(kF4Threads),
                         0, st, q, s, nchunks, out);
    return hipGetLastError();
  }
  const int64_t rows = gemm_rows_per_batch, batch = rows_total / rows;
  const int steps = t4_steps(batch, rows, cols);
  const dim3 grid = t4_grid(batch, rows, cols, steps);
  if (steps == kT4Steps)
    hipLaunchKernelGGL(dequant_tiles_fp4_kernel<kT4Steps>, grid, dim3(kF4Threads), 0, st, q, s, batch, rows,
                       (int)cols, out);
  else
    hipLaunchKernelGGL(dequant_tiles_fp4_kernel<1>, grid, dim3(kF4Threads), 0, st, q, s, batch, rows,
                       (int)cols, out);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Both orientations of expert weights from one read: w [E, N, K] ->
//   q   [E, N, K/2] (blocks along K), s   GEMM layout [E][K/128][N][4]
//   q_t [E, K, N/2] (blocks along N), s_t GEMM layout [E][N/128][K][4]
// N and K multiples of 128.  A workgroup takes a 256 x 256 tile (its part
// inside [N, K]); wave w rows n0 + 32w .. +31, one block of the second
// orientation; lane l rows 32w + 16(l/32) + i and the 16-byte piece l%32 of
// each row.  A DPP quad holds a block of a row; a lane and its partner l ^ 32
// a block of a column.  The second orientation's codes go through a
// [256 k][256 n] tile of 4-bit codes in LDS, so that q_t is stored in
// 128-byte runs like q.  Tiles down the rows first, so that these runs of q_t
// lie side by side, and streaming stores: 16 x 8192 x 5120 in 356 us (5.8 TB/s),
// tiles along the rows 392, without streaming 384.
// ---------------------------------------------------------------------------
constexpr int kW4 = 256;                  // tile edge
constexpr int kW4Threads = 512;
constexpr int kW4Row = kW4 / 2;           // bytes of a code-tile row

// 8-byte slot of a code-tile row, swizzled by the column group so that the
// lanes of a wave (consecutive groups of 8 rows) spread over the banks
__device__ __forceinline__ int w4_slot(int k, int slot) { return slot ^ ((k >> 3) & 15); }

__global__ __launch_bounds__(kW4Threads) __attribute__((amdgpu_waves_per_eu(4))) void quant_weights_fp4_kernel(
    const uint16_t* __restrict__ w, int64_t N, int64_t K, uint8_t* __restrict__ q, uint8_t* __restrict__ s,
    uint8_t* __restrict__ q_t, uint8_t* __restrict__ s_t) {
  __shared__ __attribute__((aligned(16))) uint8_t codes[kW4 * kW4Row];   // [256 k][256 n], 4 bits each
  __shared__ __attribute__((aligned(16))) uint8_t srow[2 * kW4 * 4];     // [k chunk][row][4 blocks]
  __shared__ __attribute__((aligned(16))) uint8_t scol[2 * kW4 * 4];     // [n chunk][col][4 blocks]
  const int tid = threadIdx.x, wv = tid >> 6, lane = tid & 63;
  const int half = lane >> 5, pc = lane & 31;
  const int64_t b = blockIdx.z, n0 = (int64_t)blockIdx.x * kW4, k0 = (int64_t)blockIdx.y * kW4;
  const int r0 = 32 * wv + 16 * half;
  const bool k_in = k0 + 8 * pc < K;      // K % 128 == 0: a piece is wholly inside or wholly past
  const uint16_t* wb = w + b * N * K;
  v4i v[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    v[i] = (v4i){0, 0, 0, 0};
    if (k_in && n0 + r0 + i < N)
      v[i] = __builtin_nontemporal_load((const v4i*)(wb + (n0 + r0 + i) * K + k0 + 8 * pc));
  }
  const int kb = pc >> 2;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int64_t n = n0 + r0 + i;
    const uint32_t byte = e8m0_fp4_from_absbits(quad_max(absmax8(v[i])));
    if (k_in && n < N)
      __builtin_nontemporal_store(quant8_fp4(v[i], byte), (uint32_t*)(q + (b * N + n) * (K / 2) + k0 / 2 + 4 * pc));
    if ((pc & 3) == 0) srow[(kb >> 2) * (kW4 * 4) + (r0 + i) * 4 + (kb & 3)] = (uint8_t)byte;
  }
  // column amax over the 32-row block: the lane's 16 rows, then the partner's
  us2 cm[4] = {(us2){0, 0}, (us2){0, 0}, (us2){0, 0}, (us2){0, 0}};
#pragma unroll
  for (int i = 0; i < 16; ++i)
#pragma unroll
    for (int d = 0; d < 4; ++d)
      cm[d] = __builtin_elementwise_max(cm[d], __builtin_bit_cast(us2, (uint32_t)v[i][d] & 0x7FFF7FFFu));
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    const uint32_t other = (uint32_t)__shfl_xor((int)__builtin_bit_cast(uint32_t, cm[d]), 32);
    const us2 both = __builtin_elementwise_max(cm[d], __builtin_bit_cast(us2, other));
#pragma unroll
    for (int hi = 0; hi < 2; ++hi) {
      const uint32_t byte = e8m0_fp4_from_absbits(both[hi]);
      const float scale = __uint_as_float(byte << 23);
      v2i o;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        uint32_t pr[4];
#pragma unroll
        for (int u = 0; u < 4; ++u)      // column 2d + hi of two consecutive rows
          pr[u] = __builtin_amdgcn_perm((uint32_t)v[8 * j + 2 * u + 1][d], (uint32_t)v[8 * j + 2 * u][d],
                                        hi ? 0x07060302u : 0x05040100u);
        uint32_t c = cvt2_e2m1<0>(0u, pr[0], scale);
        c = cvt2_e2m1<1>(c, pr[1], scale);
        c = cvt2_e2m1<2>(c, pr[2], scale);
        c = cvt2_e2m1<3>(c, pr[3], scale);
        o[j] = byte == 0xFFu ? 0 : (int)c;
      }
      const int k = 8 * pc + 2 * d + hi;
      *(v2i*)(codes + k * kW4Row + 8 * w4_slot(k, 2 * wv + half)) = o;
      if (half == 0) scol[(wv >> 2) * (kW4 * 4) + k * 4 + (wv & 3)] = (uint8_t)byte;
    }
  }
  __syncthreads();
  // q_t: 16 bytes (two slots, 32 rows) per thread and step, 8 threads a row
#pragma unroll
  for (int it = 0; it < kW4 * 8 / kW4Threads; ++it) {
    const int k = tid / 8 + (kW4Threads / 8) * it, p = tid % 8;
    const v2i lo = *(const v2i*)(codes + k * kW4Row + 8 * w4_slot(k, 2 * p));
    const v2i hi = *(const v2i*)(codes + k * kW4Row + 8 * w4_slot(k, 2 * p + 1));
    if (k0 + k < K && n0 + 32 * p < N)
      __builtin_nontemporal_store((v4i){lo[0], lo[1], hi[0], hi[1]},
                                  (v4i*)(q_t + (b * K + k0 + k) * (N / 2) + n0 / 2 + 16 * p));
  }
  {
    const int ch = tid / kW4, r = tid % kW4;
    if (n0 + r < N && k0 + 128 * ch < K)
      *(uint32_t*)(s + b * (K / 32) * N + ((k0 >> 7) + ch) * N * 4 + (n0 + r) * 4) =
          *(const uint32_t*)(srow + ch * (kW4 * 4) + r * 4);
    if (k0 + r < K && n0 + 128 * ch < N)
      *(uint32_t*)(s_t + b * (N / 32) * K + ((n0 >> 7) + ch) * K * 4 + (k0 + r) * 4) =
          *(const uint32_t*)(scol + ch * (kW4 * 4) + r * 4);
  }
}

hipError_t launch_quant_weights_fp4(const uint16_t* w, int64_t E, int64_t N, int64_t K, uint8_t* q, uint8_t* s,
                                    uint8_t* q_t, uint8_t* s_t, hipStream_t st) {
  if (E == 0 || N == 0 || K == 0) return hipSuccess;
  const dim3 grid((unsigned)((N + kW4 - 1) / kW4), (unsigned)((K + kW4 - 1) / kW4), (unsigned)E);
  hipLaunchKernelGGL(quant_weights_fp4_kernel, grid, dim3(kW4Threads), 0, st, w, N, K, q, s, q_t, s_t);
  return hipGetLastError();
}

}  // namespace mxk
