// The router of a mixture-of-experts layer (gfx950): logits of T tokens for E
// experts -> the k experts of each token and their combine weights, and the
// gradient of the logits.
//
//   s = softmax(l) or sigmoid(l),  c = s + bias
//   value of a group of E/G experts: its largest c, or the sum of its two largest
//   expert_idx = the k largest c among the experts of the topk_groups best groups
//   combine = scale * s[expert_idx] (/ sum of s[expert_idx])
//
// Equal values go to the lowest index.  A masked expert (logit -inf or the
// lowest finite value of its type) has the score 0 and comes behind all others;
// so does one whose c is NaN.
//
// The choice is that of the scores in 64 bits.  Softmax and sigmoid are
// monotone, so without a bias (and with the groups' values being maxima) the
// logits themselves are compared, which is exact; with one, or with sums of
// two, c is computed in fp64: at fp32's 2^-24, one token in some thousand would
// have two experts (of 256) out of order.
//
// One wave per token, expert v * 64 + lane in register v of a lane: every load
// is a run of whole lines, and an expert's number follows from where it is
// found.  An arg-max is a reduction over the lanes by DPP and one ballot per
// register.  Nothing goes through LDS or memory.
#include <type_traits>

#include "mx_device.h"
#include "mx_kernels.h"

namespace mxk {

namespace {

constexpr int kRouterWaves = 4;

__device__ __forceinline__ float lane_value(float x, int lane) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), lane));
}
__device__ __forceinline__ double lane_value(double x, int lane) {
  const uint64_t u = (uint64_t)__double_as_longlong(x);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)u, lane);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), lane);
  return __longlong_as_double((long long)(((uint64_t)hi << 32) | lo));
}

// x of the lane that the DPP control names, x itself where there is none.
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp(float x) {
  const int u = __float_as_int(x);
  return __int_as_float(__builtin_amdgcn_update_dpp(u, u, CTRL, ROWS, 0xF, false));
}
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp(double x) {
  const uint64_t u = (uint64_t)__double_as_longlong(x);
  const int lo = (int)(uint32_t)u, hi = (int)(uint32_t)(u >> 32);
  const uint32_t l = (uint32_t)__builtin_amdgcn_update_dpp(lo, lo, CTRL, ROWS, 0xF, false);
  const uint32_t h = (uint32_t)__builtin_amdgcn_update_dpp(hi, hi, CTRL, ROWS, 0xF, false);
  return __longlong_as_double((long long)(((uint64_t)h << 32) | l));
}

__device__ __forceinline__ float larger(float a, float b) { return fmaxf(a, b); }
__device__ __forceinline__ double larger(double a, double b) { return fmax(a, b); }

// Largest x of the wave, in every lane.
template <class C>
__device__ __forceinline__ C wave_max(C x) {
  x = larger(x, dpp<0x111, 0xF>(x));      // row_shr:1, 2, 4, 8: lane 15 of a row has the row's
  x = larger(x, dpp<0x112, 0xF>(x));
  x = larger(x, dpp<0x114, 0xF>(x));
  x = larger(x, dpp<0x118, 0xF>(x));
  x = larger(x, dpp<0x142, 0xA>(x));      // row_bcast:15 into rows 1 and 3
  x = larger(x, dpp<0x143, 0xC>(x));      // row_bcast:31 into rows 2 and 3
  return lane_value(x, 63);
}

// Sum over the wave, in every lane, always added in the same order.
template <class C>
__device__ __forceinline__ C wave_sum(C x) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) x += __shfl_xor(x, d);
  return x;
}

template <class T>
struct Logits;
template <>
struct Logits<float> {
  static __device__ __forceinline__ float load(const float* p) { return *p; }
  static __device__ __forceinline__ void store(float* p, float x) { *p = x; }
  static constexpr float lowest = -3.402823466e38f;
};
template <>
struct Logits<uint16_t> {
  static __device__ __forceinline__ float load(const uint16_t* p) { return __uint_as_float((uint32_t)*p << 16); }
  static __device__ __forceinline__ void store(uint16_t* p, float x) { *p = (uint16_t)pack_bf16x2_rne(x, 0.f); }
  static constexpr float lowest = -3.389531390e38f;
};

// exp(x) for x <= 0: the hardware's 2^y of x / ln 2 in two parts, off by about
// 2^-23 of the result at any x.
__device__ __forceinline__ float exp_neg(float x) {
  const float y = x * 1.442695041f;
  const float lo = fmaf(x, 1.925963033e-8f, fmaf(x, 1.442695041f, -y));
  const float p = __builtin_amdgcn_exp2f(y);
  return x > -120.f ? fmaf(p * lo, 0.6931471806f, p) : x == x ? 0.f : x;
}

__device__ __forceinline__ float sigmoid(float x) {
  const float e = exp_neg(-fabsf(x));
  return (x < 0.f ? e : 1.f) / (1.f + e);
}

}  // namespace

// V registers of experts per lane; VALUES: c in fp64, else the logits decide.
template <int V, class T, bool VALUES>
__global__ __launch_bounds__(kRouterWaves * 64) void router_fwd_kernel(const T* __restrict__ logits,
                                                                       const float* __restrict__ bias, RouterArgs a) {
  typedef std::conditional_t<VALUES, double, float> C;
  constexpr C kLowest = VALUES ? (C)-1.7976931348623157e308 : (C)-3.402823466e38f;
  const int lane = threadIdx.x & 63;
  const int64_t step = (int64_t)gridDim.x * kRouterWaves;
  const int each = a.E / a.groups;
  const float kInf = __builtin_inff();
  for (int64_t t = (int64_t)blockIdx.x * kRouterWaves + (threadIdx.x >> 6); t < a.T; t += step) {
    float l[V];
    uint32_t open = 0;          // experts of this lane that may be chosen and are not yet
    uint32_t live = 0;          // ... whose logit is not masked
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = v * 64 + lane;
      l[v] = e < a.E ? Logits<T>::load(logits + t * a.E + e) : -kInf;
      if (e < a.E) open |= 1u << v;
      if (!(l[v] <= Logits<T>::lowest)) live |= 1u << v;
    }
    // largest logit and sum of exponentials of the whole row
    float top = 0.f, total = 0.f;
    double total64 = 0.;
    if (a.score == MX_SCORE_SOFTMAX && (VALUES || !a.renormalize)) {
      float m = -kInf;
#pragma unroll
      for (int v = 0; v < V; ++v) m = fmaxf(m, live >> v & 1 ? l[v] : -kInf);
      top = wave_max(m);
      top = top > -kInf ? top : 0.f;
#pragma unroll
      for (int v = 0; v < V; ++v) total += live >> v & 1 ? exp_neg(l[v] - top) : 0.f;
      total = wave_sum(total);
    }
    C c[V];
    if constexpr (VALUES) {
      double s[V];
      if (a.score == MX_SCORE_SOFTMAX) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
          s[v] = live >> v & 1 ? exp((double)l[v] - (double)top) : 0.;
          total64 += s[v];
        }
        total64 = wave_sum(total64);
#pragma unroll
        for (int v = 0; v < V; ++v) s[v] = s[v] / total64;
      } else {
#pragma unroll
        for (int v = 0; v < V; ++v) s[v] = 1. / (1. + exp(-(double)l[v]));
      }
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int e = v * 64 + lane;
        c[v] = bias != nullptr && e < a.E ? s[v] + (double)bias[e] : s[v];
      }
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) c[v] = l[v];
    }
#pragma unroll
    for (int v = 0; v < V; ++v) c[v] = (live >> v & 1) && c[v] > kLowest ? c[v] : kLowest;

    if (a.groups > 1) {
      // group g's value in lane g
      C value = -(C)kInf;
      for (int g = 0; g < a.groups; ++g) {
        C m = kLowest;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const int e = v * 64 + lane - g * each;
          if (e >= 0 && e < each) m = larger(m, c[v]);
        }
        const C first = wave_max(m);
        C second = kLowest;
        if (a.group_top2) {
          // without one holder of the largest value
          bool found = false;
#pragma unroll
          for (int v = 0; v < V; ++v) {
            const int e = v * 64 + lane - g * each;
            const bool in = e >= 0 && e < each;
            const uint64_t at = __ballot(in && c[v] == first);
            const bool mine = !found && at != 0 && __builtin_ctzll(at) == lane;
            if (in && !mine) second = larger(second, c[v]);
            found = found || at != 0;
          }
          second = wave_max(second);
        }
        if (lane == g) value = second > kLowest ? first + second : first;
      }
      uint64_t kept = 0;
      for (int j = 0; j < a.topk_groups; ++j) {
        const bool free = lane < a.groups && !(kept >> lane & 1);
        const C best = wave_max(free ? value : -(C)kInf);
        kept |= 1ull << __builtin_ctzll(__ballot(free && value == best));
      }
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int e = v * 64 + lane;
        if (!(kept >> (e / each & 63) & 1)) open &= ~(1u << v);
      }
    }

    // slot j's expert and logit in lane j
    int id = 0;
    float picked = -kInf;
    bool on = false;
    for (int j = 0; j < a.k; ++j) {
      C m = -(C)kInf;
#pragma unroll
      for (int v = 0; v < V; ++v) m = larger(m, open >> v & 1 ? c[v] : -(C)kInf);
      const C best = wave_max(m);
      bool found = false;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const uint64_t at = __ballot((open >> v & 1) && c[v] == best);
        if (!found && at != 0) {
          found = true;
          const int who = __builtin_ctzll(at);
          const float lj = lane_value(l[v], who);
          if (lane == who) open &= ~(1u << v);
          if (lane == j) {
            id = v * 64 + who;
            picked = lj;
            on = !(lj <= Logits<T>::lowest);
          }
        }
      }
    }

    // weights, slot j in lane j
    float w = 0.f;
    if (a.renormalize) {
      // relative to the largest of the slots, so that their sum is no underflow
      const float m0 = wave_max(on ? picked : -kInf);
      const float m = m0 > -kInf ? m0 : 0.f;
      if (on) {
        if (a.score == MX_SCORE_SOFTMAX) w = exp_neg(picked - m);
        else w = exp_neg(fminf(picked, 0.f) - fminf(m, 0.f)) / (1.f + exp_neg(-fabsf(picked)));
      }
      const float sum = wave_sum(w);
      w = on ? w / sum : 0.f;
      if (a.score == MX_SCORE_SOFTMAX) {
        // a NaN anywhere is one in every score of its token, chosen or not
        bool nan = false;
#pragma unroll
        for (int v = 0; v < V; ++v) nan = nan || l[v] != l[v];
        if (__ballot(nan)) w = __builtin_nanf("");
      }
    } else if (on) {
      w = a.score == MX_SCORE_SOFTMAX ? exp_neg(picked - top) / total : sigmoid(picked);
    }
    if (lane < a.k) {
      a.expert_idx[t * a.k + lane] = id;
      a.combine[t * a.k + lane] = w * a.scale;
    }
  }
}

// Gradient of the logits (see mx_topk_router_bwd).
template <int V, class T>
__global__ __launch_bounds__(kRouterWaves * 64) void router_bwd_kernel(const T* __restrict__ logits,
                                                                       const float* __restrict__ dcombine,
                                                                       RouterArgs a, T* __restrict__ dlogits) {
  const int lane = threadIdx.x & 63;
  const int64_t step = (int64_t)gridDim.x * kRouterWaves;
  const float kInf = __builtin_inff();
  for (int64_t t = (int64_t)blockIdx.x * kRouterWaves + (threadIdx.x >> 6); t < a.T; t += step) {
    // slot j in lane j
    int id = -1;
    float w = 0.f, g = 0.f;
    if (lane < a.k) {
      id = a.expert_idx[t * a.k + lane];
      w = a.combine[t * a.k + lane];
      g = dcombine[t * a.k + lane];
    }
    const float p = w / a.scale;
    float d;                                   // the slot's part of its expert's gradient
    float dot = 0.f;
    const bool dense = a.score == MX_SCORE_SOFTMAX && !a.renormalize;
    if (a.renormalize || dense) dot = wave_sum(g * p);
    if (dense) {
      d = g * a.scale;
      dot *= a.scale;
    } else if (a.renormalize) {
      d = w * (g - dot);
      if (a.score == MX_SCORE_SIGMOID && lane < a.k && id >= 0 && id < a.E)
        d *= sigmoid(-Logits<T>::load(logits + t * a.E + id));
    } else {
      d = w * (1.f - p) * g;
    }
    float out[V];
#pragma unroll
    for (int v = 0; v < V; ++v) out[v] = 0.f;
    for (int j = 0; j < a.k; ++j) {
      const int e = __builtin_amdgcn_readlane(id, j);
      const float dj = lane_value(d, j);
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (e == v * 64 + lane) out[v] += dj;
    }
    if (dense) {
      float l[V], m = -kInf, total = 0.f;
      uint32_t live = 0;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int e = v * 64 + lane;
        l[v] = e < a.E ? Logits<T>::load(logits + t * a.E + e) : -kInf;
        if (!(l[v] <= Logits<T>::lowest)) live |= 1u << v;
        m = fmaxf(m, live >> v & 1 ? l[v] : -kInf);
      }
      const float top = wave_max(m);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        l[v] = live >> v & 1 ? exp_neg(l[v] - top) : 0.f;
        total += l[v];
      }
      total = wave_sum(total);
#pragma unroll
      for (int v = 0; v < V; ++v) out[v] = live >> v & 1 ? l[v] / total * (out[v] - dot) : 0.f;
    }
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (v * 64 + lane < a.E) Logits<T>::store(dlogits + t * a.E + v * 64 + lane, out[v]);
  }
}

namespace {

// Enough workgroups for eight waves on every SIMD; they walk the tokens.
dim3 router_grid(int64_t T) {
  const int64_t n = (T + kRouterWaves - 1) / kRouterWaves;
  return dim3((unsigned)(n < 2048 ? n : 2048));
}

template <int V, class T>
hipError_t launch_fwd(const RouterArgs& a, hipStream_t st) {
  const bool values = a.bias != nullptr || (a.groups > 1 && a.group_top2);
  if (values)
    hipLaunchKernelGGL((router_fwd_kernel<V, T, true>), router_grid(a.T), dim3(kRouterWaves * 64), 0, st,
                       (const T*)a.logits, a.bias, a);
  else
    hipLaunchKernelGGL((router_fwd_kernel<V, T, false>), router_grid(a.T), dim3(kRouterWaves * 64), 0, st,
                       (const T*)a.logits, a.bias, a);
  return hipGetLastError();
}

template <int V, class T>
hipError_t launch_bwd(const RouterArgs& a, const float* dcombine, void* dlogits, hipStream_t st) {
  hipLaunchKernelGGL((router_bwd_kernel<V, T>), router_grid(a.T), dim3(kRouterWaves * 64), 0, st, (const T*)a.logits,
                     dcombine, a, (T*)dlogits);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_router_fwd(const RouterArgs& a, hipStream_t st) {
  const int v = (a.E + 63) / 64;
  if (a.logits_f32)
    return v <= 1 ? launch_fwd<1, float>(a, st) : v <= 2 ? launch_fwd<2, float>(a, st) : v <= 4 ? launch_fwd<4, float>(a, st)
           : v <= 8 ? launch_fwd<8, float>(a, st) : launch_fwd<16, float>(a, st);
  return v <= 1 ? launch_fwd<1, uint16_t>(a, st) : v <= 2 ? launch_fwd<2, uint16_t>(a, st)
         : v <= 4 ? launch_fwd<4, uint16_t>(a, st) : v <= 8 ? launch_fwd<8, uint16_t>(a, st)
                                                             : launch_fwd<16, uint16_t>(a, st);
}

hipError_t launch_router_bwd(const RouterArgs& a, const float* dcombine, void* dlogits, hipStream_t st) {
  const int v = (a.E + 63) / 64;
  if (a.logits_f32)
    return v <= 1 ? launch_bwd<1, float>(a, dcombine, dlogits, st) : v <= 2 ? launch_bwd<2, float>(a, dcombine, dlogits, st)
           : v <= 4 ? launch_bwd<4, float>(a, dcombine, dlogits, st) : v <= 8 ? launch_bwd<8, float>(a, dcombine, dlogits, st)
                                                             : launch_bwd<16, float>(a, dcombine, dlogits, st);
  return v <= 1 ? launch_bwd<1, uint16_t>(a, dcombine, dlogits, st) : v <= 2 ? launch_bwd<2, uint16_t>(a, dcombine, dlogits, st)
         : v <= 4 ? launch_bwd<4, uint16_t>(a, dcombine, dlogits, st)
         : v <= 8 ? launch_bwd<8, uint16_t>(a, dcombine, dlogits, st) : launch_bwd<16, uint16_t>(a, dcombine, dlogits, st);
}

}  // namespace mxk
