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
// router_pick_kernel serves every choice whose groups lie along lanes: L lanes per
// token, each with V consecutive experts in registers, several tokens per wave.  A
// lane sorts its experts once, as 32-bit keys (what the expert lacks to the best one,
// and its index below): then one pick is a maximum over the lanes' first keys (DPP)
// and a shift in the lane that had it.  The keys hold the logits of bf16 exactly; the
// differences of fp32 logits and of computed scores they hold to 2^-14 of themselves
// or better, so two picks that follow each other are only taken for ordered where
// their keys are further apart than that and the error of the fp32 scores; a wave
// with a token where they are not (random logits: one in some hundred) does its choice
// again in fp64.  router_walk_kernel takes groups that are no power of two of lanes: one wave
// per token, expert v * 64 + lane in register v, an arg-max per pick over all registers, c in
// fp64 where values are compared.  4096 x 160, 8 groups, top 6: 20 us, and 11 by the logits;
// 4096 x 60, 4 groups: 10.5 and 7 (along lanes 4096 x 128, 8 groups: 9.3 and 5.5).
//
// What it reads and writes is little (4096 x 256 fp32: 4.5 MB, a microsecond); the time
// is that of k dependent picks and, where values are compared, of the one token in a
// wave that goes through fp64.  4096 x 256, 8 groups, top 8: 10 - 13 us (24 with one wave
// per token and an arg-max over its registers for each pick); 65600 x 32, top 8: 7 - 9
// (54); one token 2.2; the gradients 4 - 5 and 9 - 11 us.
#include <type_traits>

#include "mx_device.h"
#include "mx_kernels.h"

namespace mxk {

namespace {

constexpr int kRouterWaves = 4;
constexpr int kBwdCells = 512;       // logits that a wave of the backward takes (one token at least)

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

// exp(x) for x < 88: the hardware's 2^y of x / ln 2 in two parts, off by about
// 2^-23 of the result at any x.
__device__ __forceinline__ float exp32(float x) {
  const float y = x * 1.442695041f;
  const float lo = fmaf(x, 1.925963033e-8f, fmaf(x, 1.442695041f, -y));
  const float p = __builtin_amdgcn_exp2f(y);
  return x > -120.f ? fmaf(p * lo, 0.6931471806f, p) : x == x ? 0.f : x;
}

__device__ __forceinline__ float sigmoid(float x) {
  const float e = exp32(-fabsf(x));
  return (x < 0.f ? e : 1.f) / (1.f + e);
}

// Over the L lanes of a token (L = 8 .. 64), in every one of them.
template <int L, class F>
__device__ __forceinline__ uint32_t over_lanes(uint32_t x, F f) {
  x = f(x, (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0xB1, 0xF, 0xF, false));      // lanes 1, then 2 apart
  x = f(x, (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x4E, 0xF, 0xF, false));
  x = f(x, (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x141, 0xF, 0xF, false));     // the other half of 8, of 16
  if (L >= 16) x = f(x, (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x140, 0xF, 0xF, false));
  if (L >= 32) {
    const auto r = __builtin_amdgcn_permlane16_swap(x, x, false, false);
    x = f(r[0], r[1]);
  }
  if (L >= 64) {
    const auto r = __builtin_amdgcn_permlane32_swap(x, x, false, false);
    x = f(r[0], r[1]);
  }
  return x;
}
template <int L>
__device__ __forceinline__ uint32_t lanes_max(uint32_t x) {
  return over_lanes<L>(x, [](uint32_t a, uint32_t b) { return max(a, b); });
}
template <int L>
__device__ __forceinline__ float lanes_max(float x) {
  return __uint_as_float(over_lanes<L>(__float_as_uint(x), [](uint32_t a, uint32_t b) {
    return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
  }));
}
template <int L>
__device__ __forceinline__ float lanes_sum(float x) {
  return __uint_as_float(over_lanes<L>(__float_as_uint(x), [](uint32_t a, uint32_t b) {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
  }));
}

// Descending sort of V keys in registers (odd-even merges).
template <int V>
__device__ __forceinline__ void sort_keys(uint32_t (&k)[V]) {
#pragma unroll
  for (int p = 1; p < V; p *= 2)
#pragma unroll
    for (int q = p; q >= 1; q /= 2)
#pragma unroll
      for (int j = q % p; j + q < V; j += 2 * q)
#pragma unroll
        for (int i = 0; i < q; ++i)
          if (i + j + q < V && (i + j) / (2 * p) == (i + j + q) / (2 * p)) {
            const uint32_t hi = max(k[i + j], k[i + j + q]);
            k[i + j + q] = min(k[i + j], k[i + j + q]);
            k[i + j] = hi;
          }
}

// V consecutive logits of a token from expert `e0` on; -inf past E.
template <int V>
__device__ __forceinline__ void load_logits(const float* row, int e0, int E, float (&l)[V]) {
  if (E % 4 == 0) {
#pragma unroll
    for (int v = 0; v < V; v += 4) {
      typedef float v4f __attribute__((ext_vector_type(4)));
      v4f x = {0.f, 0.f, 0.f, 0.f};
      const bool in = e0 + v < E;
      if (in) x = *(const v4f*)(row + e0 + v);
#pragma unroll
      for (int i = 0; i < 4; ++i) l[v + i] = in ? x[i] : -__builtin_inff();
    }
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) l[v] = e0 + v < E ? row[e0 + v] : -__builtin_inff();
  }
}
template <int V>
__device__ __forceinline__ void load_logits(const uint16_t* row, int e0, int E, float (&l)[V]) {
  if (E % 4 == 0) {
#pragma unroll
    for (int v = 0; v < V; v += 4) {
      v2i x = {0, 0};
      const bool in = e0 + v < E;
      if (in) x = *(const v2i*)(row + e0 + v);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        l[v + 2 * i] = in ? bf16lo((uint32_t)x[i]) : -__builtin_inff();
        l[v + 2 * i + 1] = in ? bf16hi((uint32_t)x[i]) : -__builtin_inff();
      }
    }
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) l[v] = e0 + v < E ? Logits<uint16_t>::load(row + e0 + v) : -__builtin_inff();
  }
}

__device__ __forceinline__ void store4(float* p, const float* x) {
  typedef float v4f __attribute__((ext_vector_type(4)));
  *(v4f*)p = (v4f){x[0], x[1], x[2], x[3]};
}
__device__ __forceinline__ void store4(uint16_t* p, const float* x) {
  *(v2i*)p = (v2i){(int)pack_bf16x2_rne(x[0], x[1]), (int)pack_bf16x2_rne(x[2], x[3])};
}

// How the picks compare.
constexpr int kExact = 0, kLogits = 1, kValues = 2;     // bf16 logits, fp32 logits, scores with bias or sums of two

}  // namespace

template <int L, int V, class T, int BY>
__global__ __launch_bounds__(kRouterWaves * 64) void router_pick_kernel(const T* __restrict__ logits,
                                                                        const float* __restrict__ bias, RouterArgs a) {
  constexpr int kSlots = MX_MOE_MAX_TOPK / L ? MX_MOE_MAX_TOPK / L : 1;      // slots a lane holds
  constexpr float kInf = __builtin_inff();
  const int sub = threadIdx.x % L;
  const int64_t token = wide_block() * (kRouterWaves * 64 / L) + threadIdx.x / L;
  const int64_t t = min(token, a.T - 1);
  const T* row = logits + t * a.E;
  const int e0 = sub * V;
  float l[V];
  load_logits<V>(row, e0, a.E, l);
  uint32_t live = 0;                              // not masked
#pragma unroll
  for (int v = 0; v < V; ++v) live |= l[v] <= Logits<T>::lowest ? 0u : 1u << v;

  // largest logit and sum of exponentials of the row
  float top = 0.f, total = 1.f;
  if (a.score == MX_SCORE_SOFTMAX && (BY == kValues || !a.renormalize)) {
    float m = -kInf;
#pragma unroll
    for (int v = 0; v < V; ++v) m = fmaxf(m, live >> v & 1 ? l[v] : -kInf);
    m = lanes_max<L>(m);
    top = m > -kInf ? m : 0.f;
    total = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) total += live >> v & 1 ? exp32(l[v] - top) : 0.f;
    total = lanes_sum<L>(total);
  }

  float c[V];
  const float inv = __builtin_amdgcn_rcpf(total);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if constexpr (BY == kValues) {
      // (2^-19 of the largest score will do)
      const float p = __builtin_amdgcn_exp2f((a.score == MX_SCORE_SOFTMAX ? l[v] - top : -l[v]) * 1.442695041f);
      const float s = a.score == MX_SCORE_SOFTMAX ? p * inv : __builtin_amdgcn_rcpf(1.f + p);
      c[v] = bias != nullptr && e0 + v < a.E ? s + bias[e0 + v] : s;
    } else {
      c[v] = l[v] + 0.f;                          // no negative zero beside a positive one
    }
    c[v] = (live >> v & 1) && c[v] > -kInf ? c[v] : -kInf;        // masked, NaN: behind the others
  }

  // Keys.  Low bits: the index, the lowest largest; 0 is no expert.
  const int bits = 32 - __builtin_clz(a.E);       // 2^bits > E
  const uint32_t low = (1u << bits) - 1;
  uint32_t key[V];
  float cmax = 0.f;
  if constexpr (BY == kExact) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const uint32_t u = __float_as_uint(c[v]);
      const uint32_t order = (u >> 16) ^ ((int)u < 0 ? 0xFFFFu : 0x8000u);
      key[v] = (c[v] > -kInf ? order << 16 : 0u) | (0xFFFFu - (uint32_t)(e0 + v));
    }
  } else {
    float m = -kInf;
#pragma unroll
    for (int v = 0; v < V; ++v) m = fmaxf(m, c[v]);
    cmax = lanes_max<L>(m);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const uint32_t lack = min(__float_as_uint(fmaxf(cmax - c[v], 0.f)), 0x7F7FFFFFu);
      const uint32_t order = max((0x7F7FFFFFu - lack) << 1 & ~low, low + 1);
      key[v] = (c[v] > -kInf ? order : 0u) | (low - (uint32_t)(e0 + v));
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) key[v] = e0 + v < a.E ? key[v] : 0u;

  // Difference below which two computed c may be out of order: scores to 2^-19 of
  // the largest of them, the sum with the bias and the difference to cmax to 2^-24.
  const float tol = BY != kValues ? 0.f : a.score == MX_SCORE_SOFTMAX ? 0x1p-17f * inv : 0x1p-20f;
  const float rel = BY == kValues ? 0x1p-22f : 0.f;
  bool unsure = BY != kExact && !(fabsf(cmax) < kInf) && cmax != -kInf;

  if (a.groups > 1) {
    // a group is n / V lanes (a power of two)
    const int n = a.E / a.groups, lanes = n / V;
    float m1 = -kInf, m2 = -kInf;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      m2 = fmaxf(m2, fminf(m1, c[v]));
      m1 = fmaxf(m1, c[v]);
    }
    for (int d = 1; d < lanes; d <<= 1) {
      const float o1 = __shfl_xor(m1, d), o2 = __shfl_xor(m2, d);
      m2 = fmaxf(fmaxf(m2, o2), fminf(m1, o1));
      m1 = fmaxf(m1, o1);
    }
    const bool two = a.group_top2 && m2 > -kInf;
    const float value = two ? m1 + m2 : m1;
    // how many groups are better, and between which numbers that lies: both c round to 2^-24
    // of themselves, which may be much more than that of a sum in which they cancel
    const float far = 2.f * tol + 5.f * rel * fabsf(m1) + (two ? 5.f * rel * fabsf(m2) : 0.f);
    const float least = value - far, most = value + far;
    const int mine = e0 / n, first = (threadIdx.x & 63) - sub;
    int better = 0, surely = 0, maybe = -1;
    for (int g = 0; g < a.groups; ++g) {
      const float o = L == 64 ? lane_value(value, g * lanes) : __shfl(value, first + g * lanes);
      better += o > value || (o == value && g < mine);
      if (BY == kValues) {
        surely += o > most;
        maybe += o >= least;
      }
    }
    // (a group of masked experts alone is behind every other for certain; a sum that leaves
    // fp32's range is not)
    unsure = unsure || (BY == kValues && e0 < a.E && m1 > -kInf &&
                        (!(fabsf(value) < kInf) ||
                         (better < a.topk_groups ? maybe >= a.topk_groups : surely < a.topk_groups)));
    if (better >= a.topk_groups) {
#pragma unroll
      for (int v = 0; v < V; ++v) key[v] = 0;
    }
  }
  sort_keys<V>(key);

  // slot r * L + sub of the token's picks in register r
  int id[kSlots];
#pragma unroll
  for (int r = 0; r < kSlots; ++r) id[r] = 0;
  uint32_t before = 0;
  auto order_of = [&](uint32_t k) { return BY == kExact ? k >> 16 : k & ~low; };
  for (int j = 0; j < (BY == kExact ? a.k : a.k + 1); ++j) {
    const uint32_t best = lanes_max<L>(key[0]);
    if constexpr (BY != kExact) {
      // the one before has to be better beyond doubt (the masked follow by index)
      const uint32_t p = order_of(before), q = order_of(best);
      const float lack_p = __uint_as_float(0x7F7FFFFFu - (p >> 1));                    // at most
      const float lack_q = __uint_as_float(0x7F7FFFFFu - ((q | low) >> 1));            // at least
      unsure = unsure || (j > 0 && q != 0 && !(lack_q > lack_p + (tol + rel * (fabsf(cmax) + lack_p))));
      before = best;
      if (j == a.k) break;
    }
    // the lane that had it moves its keys up (by masks: of selects the compiler makes
    // an index into the registers, V^2 instructions)
    const uint32_t had = key[0] == best ? ~0u : 0u;
#pragma unroll
    for (int v = 0; v + 1 < V; ++v) key[v] = (key[v] & ~had) | (key[v + 1] & had);
    key[V - 1] &= ~had;
    const int e = BY == kExact ? 0xFFFF - (int)(best & 0xFFFFu) : (int)(low - (best & low));
#pragma unroll
    for (int r = 0; r < kSlots; ++r)
      if (j == r * L + sub) id[r] = e;
  }

  if constexpr (BY != kExact) {
    if (__any(unsure)) {
      // again in fp64, an arg-max over all registers and lanes per pick
      double x[V];
      double sum = 0.;
      if (BY == kValues && a.score == MX_SCORE_SOFTMAX) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
          x[v] = live >> v & 1 ? exp((double)l[v] - (double)top) : 0.;
          sum += x[v];
        }
        for (int d = 1; d < L; d <<= 1) sum += __shfl_xor(sum, d);
      }
      constexpr double kLow = -1.7976931348623157e308;
      uint32_t open = 0;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (BY == kValues) {
          x[v] = a.score == MX_SCORE_SOFTMAX ? x[v] / sum : 1. / (1. + exp(-(double)l[v]));
          if (bias != nullptr && e0 + v < a.E) x[v] += (double)bias[e0 + v];
        } else {
          x[v] = (double)l[v] + 0.;       // as c: bits are compared below
        }
        x[v] = (live >> v & 1) && x[v] > kLow ? x[v] : kLow;
        open |= e0 + v < a.E ? 1u << v : 0u;
      }
      if (a.groups > 1) {
        const int n = a.E / a.groups, lanes = n / V;
        double m1 = kLow, m2 = kLow;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          m2 = fmax(m2, fmin(m1, x[v]));
          m1 = fmax(m1, x[v]);
        }
        for (int d = 1; d < lanes; d <<= 1) {
          const double o1 = __shfl_xor(m1, d), o2 = __shfl_xor(m2, d);
          m2 = fmax(fmax(m2, o2), fmin(m1, o1));
          m1 = fmax(m1, o1);
        }
        const double value = a.group_top2 && m2 > kLow ? m1 + m2 : m1;
        const int mine = e0 / n, first = (threadIdx.x & 63) - sub;
        int better = 0;
        for (int g = 0; g < a.groups; ++g) {
          const double o = L == 64 ? lane_value(value, g * lanes) : __shfl(value, first + g * lanes);
          better += o > value || (o == value && g < mine);
        }
        if (better >= a.topk_groups) open = 0;
      }
      // a double's bits in the order of its values, high word, low word, index
      auto high_of = [](double y) {
        const uint64_t u = (uint64_t)__double_as_longlong(y);
        return (uint32_t)(u >> 32) ^ ((int64_t)u < 0 ? 0xFFFFFFFFu : 0x80000000u);
      };
      auto low_of = [](double y) {
        const uint64_t u = (uint64_t)__double_as_longlong(y);
        return (uint32_t)u ^ ((int64_t)u < 0 ? 0xFFFFFFFFu : 0u);
      };
      for (int j = 0; j < a.k; ++j) {
        double best = kLow;
        uint32_t e = 0;                            // 1024 less the lane's best expert; 0: none left
#pragma unroll
        for (int v = V - 1; v >= 0; --v)
          if ((open >> v & 1) && x[v] >= best) {
            best = x[v];
            e = 1024u - (uint32_t)(e0 + v);
          }
        // (the reductions stand alone: every lane takes part in them)
        const uint32_t high = e ? high_of(best) : 0u, high_most = lanes_max<L>(high);
        const uint32_t lo = high == high_most ? low_of(best) : 0u, low_most = lanes_max<L>(lo);
        e = 1024u - lanes_max<L>(high == high_most && lo == low_most ? e : 0u);
        if (e >= (uint32_t)e0 && e < (uint32_t)(e0 + V)) open &= ~(1u << (e - e0));
#pragma unroll
        for (int r = 0; r < kSlots; ++r)
          if (j == r * L + sub) id[r] = (int)e;
      }
    }
  }

  // weights of the slots
  float picked[kSlots], w[kSlots];
  bool on[kSlots];
#pragma unroll
  for (int r = 0; r < kSlots; ++r) {
    const int j = r * L + sub;
    picked[r] = j < a.k ? Logits<T>::load(row + id[r]) : -kInf;
    on[r] = j < a.k && !(picked[r] <= Logits<T>::lowest);
    w[r] = 0.f;
  }
  if (a.renormalize) {
    // relative to the largest of the slots, so that their sum is no underflow
    float m = -kInf;
#pragma unroll
    for (int r = 0; r < kSlots; ++r) m = fmaxf(m, on[r] ? picked[r] : -kInf);
    m = lanes_max<L>(m);
    m = m > -kInf ? m : 0.f;
    float sum = 0.f;
#pragma unroll
    for (int r = 0; r < kSlots; ++r) {
      if (on[r])
        w[r] = a.score == MX_SCORE_SOFTMAX
                   ? exp32(picked[r] - m)
                   : exp32(fminf(picked[r], 0.f) - fminf(m, 0.f)) / (1.f + exp32(-fabsf(picked[r])));
      sum += w[r];
    }
    sum = lanes_sum<L>(sum);
    // a NaN anywhere is one in every softmax score of its token, chosen or not
    uint32_t nan = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) nan |= a.score == MX_SCORE_SOFTMAX && l[v] != l[v] ? 1u : 0u;
    nan = lanes_max<L>(nan);
#pragma unroll
    for (int r = 0; r < kSlots; ++r) w[r] = nan ? __builtin_nanf("") : on[r] ? w[r] / sum : 0.f;
  } else {
#pragma unroll
    for (int r = 0; r < kSlots; ++r)
      if (on[r]) w[r] = a.score == MX_SCORE_SOFTMAX ? exp32(picked[r] - top) / total : sigmoid(picked[r]);
  }
  if (token < a.T) {
#pragma unroll
    for (int r = 0; r < kSlots; ++r) {
      const int j = r * L + sub;
      if (j < a.k) {
        a.expert_idx[t * a.k + j] = id[r];
        a.combine[t * a.k + j] = w[r] * a.scale;
      }
    }
  }
}

// V registers of experts per lane; VALUES: c in fp64, else the logits decide.
template <int V, class T, bool VALUES>
__global__ __launch_bounds__(kRouterWaves * 64) void router_walk_kernel(const T* __restrict__ logits,
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
      for (int v = 0; v < V; ++v) total += live >> v & 1 ? exp32(l[v] - top) : 0.f;
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
        if (a.score == MX_SCORE_SOFTMAX) w = exp32(picked - m);
        else w = exp32(fminf(picked, 0.f) - fminf(m, 0.f)) / (1.f + exp32(-fabsf(picked)));
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
      w = a.score == MX_SCORE_SOFTMAX ? exp32(picked - top) / total : sigmoid(picked);
    }
    if (lane < a.k) {
      a.expert_idx[t * a.k + lane] = id;
      a.combine[t * a.k + lane] = w * a.scale;
    }
  }
}

// Gradient of the logits (see mx_topk_router_bwd).  A wave takes `n` tokens, whose
// slots and rows are runs of memory: a lane per slot, then one per token for the sum
// over its slots, then one per slot again, which adds its part to the row in LDS (the
// forward's ids are distinct: every cell gets one), and the rows leave 16 bytes a lane.
// The softmax of a row needs no sum over it: its largest slot's weight and logit give
// s[e] = p exp(l[e] - l).  65600 x 32 takes 11 us, 1.3 TB/s with the vector unit at 19%: each of
// its 4100 waves goes from the ids to the logits they name, to LDS and back three times, and is
// found waiting for one of them in 55% of its cycles (4096 x 256: 5 us, 65%).
template <class T>
__global__ __launch_bounds__(64) void router_bwd_kernel(const T* __restrict__ logits, const float* __restrict__ dcombine,
                                                        RouterArgs a, int n, T* __restrict__ dlogits) {
  extern __shared__ float lds[];
  const int lane = threadIdx.x;
  const int64_t t0 = wide_block() * n;
  if (t0 >= a.T) return;
  n = (int)min((int64_t)n, a.T - t0);
  const int slots = n * a.k, cells = n * a.E;
  float* row = lds;                               // [n][E] the chosen experts' part
  float* share = row + cells;                     // [n][k] weight over scale
  float* grad = share + slots;                    // [n][k]
  float* factor = grad + slots;                   // [n][k] what grad is multiplied with, or the logit
  int* id = (int*)(factor + slots);               // [n][k]
  float* ref = (float*)(id + slots);              // [n] sum over the slots, largest slot's logit and share
  const bool dense = a.score == MX_SCORE_SOFTMAX && !a.renormalize;
  for (int i = lane; i < slots; i += 64) {
    const int e = a.expert_idx[t0 * a.k + i];
    const float w = a.combine[t0 * a.k + i], p = w / a.scale;
    const bool in = e >= 0 && e < a.E;
    float x = w;
    if (dense || a.score == MX_SCORE_SIGMOID) {
      const float l = in ? Logits<T>::load(logits + (t0 + (uint32_t)i / (uint32_t)a.k) * a.E + e) : 0.f;
      x = l;
      if (!dense) {
        // 1 - s from the logit: of 1 - p little is left where p is close to 1 (at a logit of 10
        // it is off by 2^-11, from 17 on by all of it; the load: 3.9 us for 3.6 at 4096 x 256).
        // A weight that is not the logit's score, by more than the roundings of both, stands
        // for itself.
        float rest = sigmoid(-l);
        if (!a.renormalize && !(fabsf(rest - (1.f - p)) <= 0x1p-20f)) rest = 1.f - p;
        x = w * rest;
      }
    }
    share[i] = p;
    grad[i] = w != 0.f ? dcombine[t0 * a.k + i] : 0.f;      // none from a masked expert's slot, whatever comes in
    factor[i] = x;
    id[i] = in ? e : -1;
  }
  for (int i = lane; i < cells; i += 64) row[i] = 0.f;
  __syncthreads();
  if (a.renormalize || dense) {
    for (int t = lane; t < n; t += 64) {
      float dot = 0.f, most = 0.f, at = 0.f;
#pragma unroll 4
      for (int j = 0; j < a.k; ++j) {
        const float p = share[t * a.k + j], x = factor[t * a.k + j];
        dot = fmaf(grad[t * a.k + j], p, dot);
        const bool more = !(p <= most);
        most = more ? p : most;
        at = more ? x : at;
      }
      ref[3 * t] = dot;
      ref[3 * t + 1] = at;
      ref[3 * t + 2] = most;
    }
    __syncthreads();
  }
  for (int i = lane; i < slots; i += 64) {
    const int t = (uint32_t)i / (uint32_t)a.k;
    const float g = grad[i];
    const float x = factor[i], d = dense ? g : share[i] == 0.f ? 0.f : x * (a.renormalize ? g - ref[3 * t] : g);
    if (id[i] >= 0) atomicAdd(row + t * a.E + id[i], d);
  }
  __syncthreads();
  auto softmax_grad = [&](const float* r, float l, float g) {
    return l <= Logits<T>::lowest || r[2] == 0.f ? 0.f : exp32(l - r[1]) * r[2] * (a.scale * (g - r[0]));
  };
  const T* src = logits + t0 * a.E;
  T* dst = dlogits + t0 * a.E;
  if (a.E % 4 == 0) {
    for (int i = 4 * lane; i < cells; i += 256) {
      float o[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) o[u] = row[i + u];
      if (dense) {
        const float* p = ref + 3 * ((uint32_t)i / (uint32_t)a.E);
        const float r[3] = {p[0], p[1], p[2]};
        float l[4];
        load_logits<4>(src + i, 0, 4, l);
#pragma unroll
        for (int u = 0; u < 4; ++u) o[u] = softmax_grad(r, l[u], o[u]);
      }
      store4(dst + i, o);
    }
  } else {
    for (int i = lane; i < cells; i += 64) {
      float o = row[i];
      if (dense) o = softmax_grad(ref + 3 * ((uint32_t)i / (uint32_t)a.E), Logits<T>::load(src + i), o);
      Logits<T>::store(dst + i, o);
    }
  }
}

namespace {

// Enough workgroups for eight waves on every SIMD; they walk the tokens.
dim3 router_grid(int64_t T) {
  const int64_t n = (T + kRouterWaves - 1) / kRouterWaves;
  return dim3((unsigned)(n < 2048 ? n : 2048));
}

// A wave per token, for groups that do not lie along lanes.
template <int V, class T>
hipError_t launch_walk(const RouterArgs& a, hipStream_t st) {
  if (a.bias != nullptr || a.group_top2)
    hipLaunchKernelGGL((router_walk_kernel<V, T, true>), router_grid(a.T), dim3(kRouterWaves * 64), 0, st,
                       (const T*)a.logits, a.bias, a);
  else
    hipLaunchKernelGGL((router_walk_kernel<V, T, false>), router_grid(a.T), dim3(kRouterWaves * 64), 0, st,
                       (const T*)a.logits, a.bias, a);
  return hipGetLastError();
}

template <class T>
hipError_t launch_bwd(const RouterArgs& a, const float* dcombine, void* dlogits, hipStream_t st) {
  const int n = a.E <= kBwdCells / 64 ? 64 : a.E < kBwdCells ? kBwdCells / a.E : 1;
  const size_t bytes = (size_t)n * (a.E + 4 * a.k + 3) * sizeof(float);
  hipLaunchKernelGGL((router_bwd_kernel<T>), wide_grid((a.T + n - 1) / n), dim3(64), bytes, st, (const T*)a.logits,
                     dcombine, a, n, (T*)dlogits);
  return hipGetLastError();
}

}  // namespace

namespace {

// Whether scores have to be compared: added to a bias, or to each other.
bool by_values(const RouterArgs& a) { return a.bias != nullptr || (a.groups > 1 && a.group_top2); }

// Whether every group is a power of two of lanes with V experts each.
bool along_lanes(const RouterArgs& a, int V) {
  const int n = a.E / a.groups;
  return a.groups == 1 || (n % V == 0 && (n / V & (n / V - 1)) == 0);
}

template <int L, int V, class T>
hipError_t launch_pick(const RouterArgs& a, hipStream_t st) {
  constexpr int by = std::is_same_v<T, float> ? kLogits : kExact;
  const int64_t per = kRouterWaves * 64 / L;
  const dim3 grid = wide_grid((a.T + per - 1) / per), block(kRouterWaves * 64);
  if (by_values(a))
    hipLaunchKernelGGL((router_pick_kernel<L, V, T, kValues>), grid, block, 0, st, (const T*)a.logits, a.bias, a);
  else
    hipLaunchKernelGGL((router_pick_kernel<L, V, T, by>), grid, block, 0, st, (const T*)a.logits, a.bias, a);
  return hipGetLastError();
}

template <class T>
hipError_t launch_fwd(const RouterArgs& a, hipStream_t st) {
  // Four experts a lane and as many lanes as that takes, so that few tokens share a wave:
  // it waits for the one of them whose choice fp32 does not decide.
  if (a.E <= 32 && along_lanes(a, 4)) return launch_pick<8, 4, T>(a, st);
  if (a.E <= 64 && along_lanes(a, 4)) return launch_pick<16, 4, T>(a, st);
  if (a.E <= 128 && along_lanes(a, 4)) return launch_pick<32, 4, T>(a, st);
  // (bf16 logits alone have no fp64 pass to wait for: half the lanes, 16384 x 256 8.1 us for 10.4)
  if (std::is_same_v<T, uint16_t> && !by_values(a) && a.E > 128 && a.E <= 256 && along_lanes(a, 8))
    return launch_pick<32, 8, T>(a, st);
  if (a.E <= 256 && along_lanes(a, 4)) return launch_pick<64, 4, T>(a, st);
  if (a.E <= 512 && along_lanes(a, 8)) return launch_pick<64, 8, T>(a, st);
  if (a.E <= 1024 && along_lanes(a, 16)) return launch_pick<64, 16, T>(a, st);
  const int v = (a.E + 63) / 64;
  return v <= 1 ? launch_walk<1, T>(a, st) : v <= 2 ? launch_walk<2, T>(a, st) : v <= 4 ? launch_walk<4, T>(a, st)
         : v <= 8 ? launch_walk<8, T>(a, st) : launch_walk<16, T>(a, st);
}

}  // namespace

hipError_t launch_router_fwd(const RouterArgs& a, hipStream_t st) {
  return a.logits_f32 ? launch_fwd<float>(a, st) : launch_fwd<uint16_t>(a, st);
}

hipError_t launch_router_bwd(const RouterArgs& a, const float* dcombine, void* dlogits, hipStream_t st) {
  return a.logits_f32 ? launch_bwd<float>(a, dcombine, dlogits, st) : launch_bwd<uint16_t>(a, dcombine, dlogits, st);
}

}  // namespace mxk
