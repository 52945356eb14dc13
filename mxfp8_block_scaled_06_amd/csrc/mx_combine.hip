// The weighted sum over a token's experts, and its gradients (gfx950):
//
//   out[t] = bf16(sum_j combine[t, j] * y[t, j])      fp32, in slot order
//   dy[t, j] = combine[t, j] * dout[t],  dcombine[t, j] = sum_n dout[t, n] y[t, j, n]
//
// y [T, k, N] bf16 or fp32.  An item (t, j) whose entry of pos is negative was not
// routed: its row of y is not read, its gradients are 0.  Streaming passes, bound by
// HBM: forward k + 1 rows of a token, backward 2k + 1 (k = 8, bf16: 16 + 2 and 32 +
// 2 bytes per column).
#include <type_traits>

#include "mx_device.h"
#include "mx_kernels.h"

namespace mxk {

namespace {

constexpr int kThreads = 256;
constexpr int kSlots = 4;      // slots whose loads go out together

// Eight values of a row.
template <class Y>
struct Eight;
template <>
struct Eight<uint16_t> {
  v4i w;
  __device__ __forceinline__ void load(const uint16_t* p) { w = __builtin_nontemporal_load((const v4i*)p); }
  __device__ __forceinline__ void zero() { w = (v4i){0, 0, 0, 0}; }
  __device__ __forceinline__ float operator[](int i) const {
    const uint32_t u = (uint32_t)w[i >> 1];
    return i & 1 ? bf16hi(u) : bf16lo(u);
  }
};
template <>
struct Eight<float> {
  v4i a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = __builtin_nontemporal_load((const v4i*)p);
    b = __builtin_nontemporal_load((const v4i*)p + 1);
  }
  __device__ __forceinline__ void zero() { a = b = (v4i){0, 0, 0, 0}; }
  __device__ __forceinline__ float operator[](int i) const { return __int_as_float(i < 4 ? a[i & 3] : b[i & 3]); }
};

__device__ __forceinline__ void store8(uint16_t* p, const float* x) {
  *(v4i*)p = (v4i){(int)pack_bf16x2_rne(x[0], x[1]), (int)pack_bf16x2_rne(x[2], x[3]),
                   (int)pack_bf16x2_rne(x[4], x[5]), (int)pack_bf16x2_rne(x[6], x[7])};
}
__device__ __forceinline__ void store8(float* p, const float* x) {
  typedef float v4f __attribute__((ext_vector_type(4)));
  *(v4f*)p = (v4f){x[0], x[1], x[2], x[3]};
  *((v4f*)p + 1) = (v4f){x[4], x[5], x[6], x[7]};
}

}  // namespace

// One thread per eight columns of a token.
template <class Y>
__global__ __launch_bounds__(kThreads) void combine_fwd_kernel(const Y* __restrict__ y, const float* __restrict__ combine,
                                                               const int32_t* __restrict__ pos, int64_t chunks, int k,
                                                               int64_t N, uint16_t* __restrict__ out) {
  const int64_t i = wide_block() * kThreads + threadIdx.x;
  if (i >= chunks) return;
  const int64_t per_row = N / 8;
  const int64_t t = chunks <= (int64_t)UINT32_MAX ? (int64_t)((uint32_t)i / (uint32_t)per_row) : i / per_row;
  const int64_t c = (i - t * per_row) * 8;
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int j0 = 0; j0 < k; j0 += kSlots) {
    Eight<Y> x[kSlots];
    float w[kSlots];
    bool on[kSlots];
#pragma unroll
    for (int j = 0; j < kSlots; ++j) {
      const int64_t item = t * k + min(j0 + j, k - 1);
      on[j] = j0 + j < k && (pos == nullptr || pos[item] >= 0);
      w[j] = combine[item];
      x[j].zero();
      if (on[j]) x[j].load(y + item * N + c);
    }
#pragma unroll
    for (int j = 0; j < kSlots; ++j)
#pragma unroll
      for (int u = 0; u < 8; ++u) acc[u] = on[j] ? fmaf(w[j], x[j][u], acc[u]) : acc[u];
  }
  store8(out + t * N + c, acc);
}

// One workgroup per token and four slots.
template <class Y>
__global__ __launch_bounds__(kThreads) void combine_bwd_kernel(const Y* __restrict__ y, const float* __restrict__ combine,
                                                               const int32_t* __restrict__ pos,
                                                               const uint16_t* __restrict__ dout, int64_t T, int k,
                                                               int64_t N, Y* __restrict__ dy,
                                                               float* __restrict__ dcombine) {
  __shared__ float part[kThreads / 64][kSlots];
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  const int64_t t = wide_block();
  if (t >= T) return;
  const int j0 = (int)blockIdx.z * kSlots, n = min(kSlots, k - j0);
  float w[kSlots], dot[kSlots];
  bool on[kSlots];
#pragma unroll
  for (int j = 0; j < kSlots; ++j) {
    const int64_t item = t * k + min(j0 + j, k - 1);
    on[j] = j < n && (pos == nullptr || pos[item] >= 0);
    w[j] = combine[item];
    dot[j] = 0.f;
  }
  for (int64_t c = tid * 8; c < N; c += kThreads * 8) {
    Eight<uint16_t> d;
    d.load(dout + t * N + c);
    Eight<Y> x[kSlots];
#pragma unroll
    for (int j = 0; j < kSlots; ++j) {
      x[j].zero();
      if (on[j] && dcombine) x[j].load(y + (t * k + j0 + j) * N + c);
    }
#pragma unroll
    for (int j = 0; j < kSlots; ++j) {
      if (j >= n) continue;
      float o[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        dot[j] = fmaf(d[u], x[j][u], dot[j]);
        o[u] = on[j] ? w[j] * d[u] : 0.f;
      }
      if (dy) store8(dy + (t * k + j0 + j) * N + c, o);
    }
  }
  if (!dcombine) return;
#pragma unroll
  for (int j = 0; j < kSlots; ++j) {
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) dot[j] += __shfl_xor(dot[j], s);
    if (lane == 0) part[wv][j] = dot[j];
  }
  __syncthreads();
  if (tid < n) {
    float sum = 0.f;
#pragma unroll
    for (int v = 0; v < kThreads / 64; ++v) sum += part[v][tid];
    bool routed = pos == nullptr || pos[t * k + j0 + tid] >= 0;
    dcombine[t * k + j0 + tid] = routed ? sum : 0.f;
  }
}

hipError_t launch_combine_fwd(const CombineArgs& a, uint16_t* out, hipStream_t st) {
  const int64_t chunks = a.T * (a.N / 8);
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

hipError_t launch_combine_bwd(const CombineArgs& a, const uint16_t* dout, void* dy, float* dcombine, hipStream_t st) {
  if (a.T == 0) return hipSuccess;
  dim3 grid = wide_grid(a.T);
  grid.z = (unsigned)((a.k + kSlots - 1) / kSlots);
  if (a.y_f32)
    hipLaunchKernelGGL(combine_bwd_kernel<float>, grid, dim3(kThreads), 0, st, (const float*)a.y, a.combine, a.pos, dout,
                       a.T, a.k, a.N, (float*)dy, dcombine);
  else
    hipLaunchKernelGGL(combine_bwd_kernel<uint16_t>, grid, dim3(kThreads), 0, st, (const uint16_t*)a.y, a.combine, a.pos,
                       dout, a.T, a.k, a.N, (uint16_t*)dy, dcombine);
  return hipGetLastError();
}

}  // namespace mxk
