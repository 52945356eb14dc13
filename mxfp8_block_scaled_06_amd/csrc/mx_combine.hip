// The weighted sum over a token's experts, and its gradients (gfx950):
//
//   out[t] = bf16(sum_j combine[t, j] * y[t, j])      fp32, in slot order
//   dy[t, j] = combine[t, j] * dout[t],  dcombine[t, j] = sum_n dout[t, n] y[t, j, n]
//
// y [T, k, N] bf16 or fp32.  An item (t, j) whose entry of pos is negative was not
// routed: its row of y is not read, its gradients are 0.  Streaming passes, bound by
// HBM: forward k + 1 rows of a token, backward 2k + 1 (k = 8, bf16: 16 + 2 and 32 +
// 2 bytes per column).  The k rows go past the caches, 16 bytes a lane, so that a
// wave's load or store is one run of 1 KiB (fp32 at 32 bytes a lane wrote half lines:
// 79 us instead of 62 for the backward below); the token's own row, which was just
// written or is read next, goes through them.  T x k x N, forward and backward:
//   8192 x 8 x 7168 bf16   173 us (6.1 TB/s)   360 us (5.5 TB/s; over the same tensors again 337)
//   16384 x 2 x 7168 bf16  104 us (6.8 TB/s)   170 us (6.9 TB/s)
//   2047 x 4 x 5120 fp32    31 us (5.5 TB/s)    61 us (5.5 TB/s)
#include <type_traits>

#include "mx_device.h"
#include "mx_kernels.h"

namespace mxk {

namespace {

constexpr int kThreads = 256;

// Sixteen bytes of a row: eight columns of bf16, four of fp32.
template <class Y>
constexpr int kCols = 16 / (int)sizeof(Y);

template <int C>
using Halves = std::conditional_t<C == 8, v4i, v2i>;   // C columns of bf16

template <class V>
__device__ __forceinline__ float half_at(V w, int i) {
  const uint32_t u = (uint32_t)w[i >> 1];
  return i & 1 ? bf16hi(u) : bf16lo(u);
}
__device__ __forceinline__ float column(v4i w, int i, const uint16_t*) { return half_at(w, i); }
__device__ __forceinline__ float column(v4i w, int i, const float*) { return __int_as_float(w[i]); }

template <int C>
__device__ __forceinline__ Halves<C> pack_halves(const float* x) {
  Halves<C> o;
#pragma unroll
  for (int i = 0; i < C / 2; ++i) o[i] = (int)pack_bf16x2_rne(x[2 * i], x[2 * i + 1]);
  return o;
}
__device__ __forceinline__ v4i pack_columns(const float* x, const uint16_t*) { return pack_halves<8>(x); }
__device__ __forceinline__ v4i pack_columns(const float* x, const float*) {
  return (v4i){__float_as_int(x[0]), __float_as_int(x[1]), __float_as_int(x[2]), __float_as_int(x[3])};
}

}  // namespace

// One thread per 16 bytes of a token's rows, four slots' loads at a time.
template <class Y>
__global__ __launch_bounds__(kThreads) void combine_fwd_kernel(const Y* __restrict__ y, const float* __restrict__ combine,
                                                               const int32_t* __restrict__ pos, int64_t chunks, int k,
                                                               int64_t N, uint16_t* __restrict__ out) {
  const int64_t i = wide_block() * kThreads + threadIdx.x;
  if (i >= chunks) return;
  constexpr int C = kCols<Y>, kSlots = 4;
  const int64_t per_row = N / C;
  const int64_t t = chunks <= (int64_t)UINT32_MAX ? (int64_t)((uint32_t)i / (uint32_t)per_row) : i / per_row;
  const int64_t c = (i - t * per_row) * C;
  float acc[C] = {};
  for (int j0 = 0; j0 < k; j0 += kSlots) {
    v4i x[kSlots];
    float w[kSlots];
    bool on[kSlots];
#pragma unroll
    for (int j = 0; j < kSlots; ++j) {
      const int64_t item = t * k + min(j0 + j, k - 1);
      on[j] = j0 + j < k && (pos == nullptr || pos[item] >= 0);
      w[j] = combine[item];
      x[j] = (v4i){0, 0, 0, 0};
      if (on[j]) x[j] = __builtin_nontemporal_load((const v4i*)(y + item * N + c));
    }
#pragma unroll
    for (int j = 0; j < kSlots; ++j)
#pragma unroll
      for (int u = 0; u < C; ++u) acc[u] = on[j] ? fmaf(w[j], column(x[j], u, y), acc[u]) : acc[u];
  }
  *(Halves<C>*)(out + t * N + c) = pack_halves<C>(acc);
}

// One workgroup of W threads per token and S slots: all slots together up to eight, so
// that dout is read once (4 a workgroup: 425 us instead of 373 for 8192 x 8 x 7168).
// From three slots on 512 threads (8192 x 8 x 7168: 337 us, 351 with 256; 2047 x 4 x
// 5120 fp32: 62 and 65); a token with fewer is too short for them (16384 x 1 x 5120:
// 82 us, 74 with 256).  Short rows leave part of the 512 without a column and would be
// faster with 256: at eight slots of bf16 and N = 512, 1024, 2048, 4096 it is 110 us for 59,
// 118 for 87, 178 for 182 and 183 for 180 (T 16384, at 4096 8192), at four slots and N =
// 1024, 2048 64 for 49 and 99 for 88; of fp32 at N = 512 111 for 87, level from 1024 on.
template <class Y, int S, int W>
__global__ __launch_bounds__(W) void combine_bwd_kernel(const Y* __restrict__ y, const float* __restrict__ combine,
                                                        const int32_t* __restrict__ pos,
                                                        const uint16_t* __restrict__ dout, int64_t T, int k,
                                                        int64_t N, Y* __restrict__ dy,
                                                        float* __restrict__ dcombine) {
  constexpr int C = kCols<Y>;
  __shared__ float part[W / 64][S];
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  const int64_t t = wide_block();
  if (t >= T) return;
  const int j0 = (int)blockIdx.z * S, n = min(S, k - j0);
  float w[S], dot[S];
  bool on[S];
#pragma unroll
  for (int j = 0; j < S; ++j) {
    const int64_t item = t * k + min(j0 + j, k - 1);
    on[j] = j < n && (pos == nullptr || pos[item] >= 0);
    w[j] = combine[item];
    dot[j] = 0.f;
  }
  for (int64_t c = tid * C; c < N; c += W * C) {
    const Halves<C> d = *(const Halves<C>*)(dout + t * N + c);
    v4i x[S];
#pragma unroll
    for (int j = 0; j < S; ++j) {
      x[j] = (v4i){0, 0, 0, 0};
      if (on[j] && dcombine) x[j] = __builtin_nontemporal_load((const v4i*)(y + (t * k + j0 + j) * N + c));
    }
#pragma unroll
    for (int j = 0; j < S; ++j) {
      if (j >= n) continue;
      float o[C];
#pragma unroll
      for (int u = 0; u < C; ++u) {
        dot[j] = fmaf(half_at(d, u), column(x[j], u, y), dot[j]);
        o[u] = on[j] ? w[j] * half_at(d, u) : 0.f;
      }
      if (dy) __builtin_nontemporal_store(pack_columns(o, y), (v4i*)(dy + (t * k + j0 + j) * N + c));
    }
  }
  if (!dcombine) return;
#pragma unroll
  for (int j = 0; j < S; ++j) {
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) dot[j] += __shfl_xor(dot[j], s);
    if (lane == 0) part[wv][j] = dot[j];
  }
  __syncthreads();
  if (tid < n) {
    float sum = 0.f;
#pragma unroll
    for (int v = 0; v < W / 64; ++v) sum += part[v][tid];
    bool routed = pos == nullptr || pos[t * k + j0 + tid] >= 0;
    dcombine[t * k + j0 + tid] = routed ? sum : 0.f;
  }
}

hipError_t launch_combine_fwd(const CombineArgs& a, uint16_t* out, hipStream_t st) {
  const int64_t chunks = a.T * (a.N / (a.y_f32 ? kCols<float> : kCols<uint16_t>));
  if (chunks == 0) return hipSuccess;
  const dim3 grid = wide_grid((chunks + kThreads - 1) / kThreads);
  if (a.y_f32)
    hipLaunchKernelGGL(combine_fwd_kernel<float>, grid, dim3(kThreads), 0, st, (const float*)a.y, a.combine, a.pos, chunks,
                       a.k, a.N, out);
  else
    hipLaunchKernelGGL(combine_fwd_kernel<uint16_t>, grid, dim3(kThreads), 0, st, (const uint16_t*)a.y, a.combine, a.pos,
                       chunks, a.k, a.N, out);
  return hipGetLastError();
}

template <class Y, int S, int W>
static void combine_bwd_grid(const CombineArgs& a, const uint16_t* dout, void* dy, float* dcombine, hipStream_t st) {
  dim3 grid = wide_grid(a.T);
  grid.z = (unsigned)((a.k + S - 1) / S);
  hipLaunchKernelGGL((combine_bwd_kernel<Y, S, W>), grid, dim3(W), 0, st, (const Y*)a.y, a.combine, a.pos, dout, a.T,
                     a.k, a.N, (Y*)dy, dcombine);
}

template <class Y>
static void combine_bwd_slots(const CombineArgs& a, const uint16_t* dout, void* dy, float* dcombine, hipStream_t st) {
  if (a.k > 4)
    combine_bwd_grid<Y, 8, 512>(a, dout, dy, dcombine, st);
  else if (a.k > 2)
    combine_bwd_grid<Y, 4, 512>(a, dout, dy, dcombine, st);
  else
    combine_bwd_grid<Y, 2, 256>(a, dout, dy, dcombine, st);
}

hipError_t launch_combine_bwd(const CombineArgs& a, const uint16_t* dout, void* dy, float* dcombine, hipStream_t st) {
  if (a.T == 0) return hipSuccess;
  if (a.y_f32)
    combine_bwd_slots<float>(a, dout, dy, dcombine, st);
  else
    combine_bwd_slots<uint16_t>(a, dout, dy, dcombine, st);
  return hipGetLastError();
}

}  // namespace mxk
