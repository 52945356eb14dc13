// A whole gated mixture-of-experts layer for a few tokens (gfx950):
//
//   g, u = MX8(x[t]) W13[e]^T    (gate rows 0..N-1, up rows N..2N-1 of W13[e])
//   h    = MX8(silu(g) * u)
//   out[t] = bf16(sum_j combine[t, j] * (h_j W2[e_j]^T))
//
// over the experts e = expert_idx[t, j] of token t, W13 [E, 2N, K] and W2
// [E, K, N] in MXFP4 or MXFP8, MX8 the MXFP8 quantization of the grouped path
// (1x32 blocks along the contraction).
//
// With a few tokens the layer is the reading of the hit experts' weights:
// every weight byte is read once, by one workgroup, straight from memory into
// the registers of the matrix instruction, and 16 tokens cost no more of them
// than one.  Two kernels, since the down projection needs all of h; grouping,
// quantization and the weighted sum happen inside them:
//   moe_gate_up_kernel  32 gate and 32 up rows of one hit expert per
//                       workgroup (one block of h), for all its tokens;
//   moe_down_kernel     16 output columns per workgroup, all hit experts, all
//                       tokens; the sum over a token's experts stays in fp32
//                       registers, so nothing is added through memory and the
//                       order of additions is fixed.
// Both split their contraction over the eight waves of the workgroup and add
// the partial sums in wave order.
//
// Matrix operand layout (v_mfma_scale_f32_16x16x128_f8f6f4): lane l holds row
// l%16, group g = l/16: E2M1 elements 32g..32g+31 in 16 bytes, E4M3 the
// 16-byte pieces g and g+4; its scale byte is block g's; its accumulators are
// column l%16, rows 4g..4g+3.  Weights are the first operand (rows), tokens
// the second (columns).
#include <algorithm>

#include "mx_device.h"
#include "mx_kernels.h"

namespace mxk {

typedef float v4f __attribute__((ext_vector_type(4)));

constexpr int kMoeWaves = 8, kMoeThreads = kMoeWaves * 64;
constexpr int kMoeRows = 32;                       // rows of h per workgroup: one scale block
constexpr int kMoeItems = kMoeMaxTokens * kMoeMaxTopk;
constexpr int kFmtE4M3 = 0, kFmtE2M1 = 4;          // the instruction's operand formats

__device__ __forceinline__ int uni(int v) { return __builtin_amdgcn_readfirstlane(v); }

// ids of the call in LDS, and the set of experts that any of them names.
// Ids outside [0, E) name none.
__device__ __forceinline__ void load_ids(const MoeArgs& a, int* s_ids, uint32_t* s_bits) {
  const int tid = threadIdx.x, n = a.T * a.topk;
  if (tid < kMaxExperts / 32) s_bits[tid] = 0u;
  __syncthreads();
  for (int i = tid; i < n; i += kMoeThreads) {
    const int e = a.ids[i];
    s_ids[i] = e;
    if (e >= 0 && e < a.E) atomicOr(&s_bits[e >> 5], 1u << (e & 31));
  }
  __syncthreads();
}

// Hit experts in ascending order: how many there are, and with them how many
// come before this lane's 32 (lanes 0..31).
__device__ __forceinline__ int count_hit(const uint32_t* s_bits, uint32_t& word, int& before) {
  const int lane = threadIdx.x & 63;
  word = lane < kMaxExperts / 32 ? s_bits[lane] : 0u;
  int incl = __popc(word);
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int v = __shfl_up(incl, d);
    if (lane >= d) incl += v;
  }
  before = incl - __popc(word);
  return uni(__shfl(incl, 63));
}

// First slot of token t that names expert e (or -1), and the sum of the
// combine weights of all its slots that do: a token that names an expert twice
// is one row of that expert.
__device__ __forceinline__ int slot_of(const int* s_ids, int t, int topk, int e) {
  int found = -1;
  for (int j = topk - 1; j >= 0; --j)
    if (s_ids[t * topk + j] == e) found = j;
  return found;
}

// 16 bytes of E2M1 or two 16-byte pieces of E4M3 of a weight row's chunk.
template <int WF>
__device__ __forceinline__ v8i load_weight(const uint8_t* row, int ch, int g) {
  if (WF == kFmtE2M1) {
    const v4i w = __builtin_nontemporal_load((const v4i*)(row + (int64_t)ch * 64 + 16 * g));
    return (v8i){w[0], w[1], w[2], w[3], 0, 0, 0, 0};
  }
  const v4i w = __builtin_nontemporal_load((const v4i*)(row + (int64_t)ch * 128 + 16 * g));
  const v4i v = __builtin_nontemporal_load((const v4i*)(row + (int64_t)ch * 128 + 64 + 16 * g));
  return (v8i){w[0], w[1], w[2], w[3], v[0], v[1], v[2], v[3]};
}

template <int WF>
__device__ __forceinline__ v4f mfma(const v8i& w, int ws, const v8i& x, int xs, const v4f& c) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, c, WF, kFmtE4M3, 0, ws, 0, xs);
}

// The lane's part of 128 bf16 values of its token in MXFP8: pieces g and g+4
// (w: 16 + 16 values) and the scale byte of block g.  Piece p belongs to block
// p/2, so a block's amax takes the neighbouring group's lane too.
__device__ __forceinline__ v8i quantize_operand(const v4i w[4], int lane, int& scale) {
  const int g = lane >> 4, l16 = lane & 15;
  uint32_t lo = max(absmax8(w[0]), absmax8(w[1])), hi = max(absmax8(w[2]), absmax8(w[3]));
  uint32_t both = lo | hi << 16;       // |bf16| bits fit 15 bits
  const uint32_t other = (uint32_t)__shfl_xor((int)both, 16);
  lo = max(lo, other & 0xFFFFu);
  hi = max(hi, other >> 16);
  const uint32_t blo = e8m0_from_absbits(lo), bhi = e8m0_from_absbits(hi);
  const float mlo = inv_scale_from_e8m0(blo == 0xFFu ? 127u : blo);
  const float mhi = inv_scale_from_e8m0(bhi == 0xFFu ? 127u : bhi);
  v8i q;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const v2i c = quant8(w[i], i < 2 ? mlo : mhi);
    const bool nan = (i < 2 ? blo : bhi) == 0xFFu;
    q[2 * i] = nan ? 0x7F7F7F7F : c[0];
    q[2 * i + 1] = nan ? 0x7F7F7F7F : c[1];
  }
  // block 0: low half of groups 0, 1; block 1: of 2, 3; blocks 2, 3: high half
  const int src = g == 1 ? l16 + 32 : g == 2 ? l16 : lane;
  const uint32_t bytes = (uint32_t)__shfl((int)(blo | bhi << 8), src);
  scale = (int)(g < 2 ? bytes & 0xFFu : bytes >> 8);
  return q;
}

// ---------------------------------------------------------------------------
// Gate and up projection, SwiGLU and the quantization of h.  Workgroup
// (n-block, hit expert): up to 16 * CT tokens of that expert.
// ---------------------------------------------------------------------------
template <int WF, int CT>
__global__ __launch_bounds__(kMoeThreads) void moe_gate_up_kernel(MoeArgs a) {
  __shared__ int s_ids[kMoeItems];
  __shared__ uint32_t s_bits[kMaxExperts / 32];
  __shared__ int s_item[kMoeMaxTokens];
  __shared__ v4f part[kMoeWaves][4][64];
  load_ids(a, s_ids, s_bits);
  const int tid = threadIdx.x, lane = tid & 63, wv = uni(tid >> 6), l16 = lane & 15, g = lane >> 4;
  uint32_t word;
  int before;
  const int hit = count_hit(s_bits, word, before);
  const int slot = blockIdx.y;
  if (slot >= hit) return;
  // the slot-th hit expert
  const uint64_t owner = __ballot(slot >= before && slot < before + __popc(word));
  const int src = __builtin_ctzll(owner);
  uint32_t w = (uint32_t)__shfl((int)word, src);
  for (int i = slot - __shfl(before, src); i > 0; --i) w &= w - 1u;
  const int e = uni(src * 32 + __builtin_ctz(w));
  // its tokens, in order: item = t * topk + slot
  int m = 0;
#pragma unroll
  for (int t0 = 0; t0 < kMoeMaxTokens; t0 += 64) {
    const int t = t0 + lane;
    const int j = t < a.T ? slot_of(s_ids, t, a.topk, e) : -1;
    const uint64_t mask = __ballot(j >= 0);
    if (wv == 0 && j >= 0) s_item[m + __builtin_popcountll(mask & ((1ull << lane) - 1))] = t * a.topk + j;
    m += __builtin_popcountll(mask);
  }
  __syncthreads();
  m = uni(m);
  const int nct = (m + 15) / 16;
  const int64_t K = a.K, N = a.N, n0 = (int64_t)blockIdx.x * kMoeRows;
  const int64_t ldw = WF == kFmtE2M1 ? K / 2 : K;
  const uint8_t* wrow[4];
  const uint8_t* srow[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int64_t n = (r < 2 ? n0 : N + n0) + 16 * (r & 1) + l16;
    wrow[r] = a.q13 + ((int64_t)e * 2 * N + n) * ldw;
    srow[r] = a.s13 + (int64_t)e * 2 * N * (K / 32) + n * 4 + g;
  }
  const uint16_t* xrow[CT];
  bool have[CT];
#pragma unroll
  for (int c = 0; c < CT; ++c) {
    have[c] = 16 * c + l16 < m;
    xrow[c] = a.x + (int64_t)(have[c] ? s_item[16 * c + l16] / a.topk : 0) * K;
  }
  v4f acc[4][CT];
#pragma unroll
  for (int r = 0; r < 4; ++r)
#pragma unroll
    for (int c = 0; c < CT; ++c) acc[r][c] = (v4f){0.f, 0.f, 0.f, 0.f};
  const int nch = (int)(K / 128), per = (nch + kMoeWaves - 1) / kMoeWaves;
  const int end = min((wv + 1) * per, nch);
  for (int ch = wv * per; ch < end; ++ch) {
    v8i wq[4];
    int ws[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      wq[r] = load_weight<WF>(wrow[r], ch, g);
      ws[r] = srow[r][(int64_t)ch * 2 * N * 4];
    }
#pragma unroll
    for (int c = 0; c < CT; ++c) {
      if (c >= nct) continue;
      v4i xw[4] = {(v4i){0, 0, 0, 0}, (v4i){0, 0, 0, 0}, (v4i){0, 0, 0, 0}, (v4i){0, 0, 0, 0}};
      if (have[c]) {
        const v4i* p = (const v4i*)(xrow[c] + ch * 128 + 16 * g);
        xw[0] = p[0];
        xw[1] = p[1];
        xw[2] = p[8];        // 64 values on
        xw[3] = p[9];
      }
      int xs;
      const v8i xq = quantize_operand(xw, lane, xs);
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[r][c] = mfma<WF>(wq[r], ws[r], xq, xs, acc[r][c]);
    }
  }
  for (int c = 0; c < CT; ++c) {
    if (c >= nct) break;
    __syncthreads();
#pragma unroll
    for (int r = 0; r < 4; ++r) part[wv][r][lane] = acc[r][c];
    __syncthreads();
    if (wv != 0) continue;
    v4f s[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      s[r] = part[0][r][lane];
#pragma unroll
      for (int v = 1; v < kMoeWaves; ++v) s[r] += part[v][r][lane];
    }
    // h of rows 4g..4g+3 and 16 + 4g..; quantized from fp32, with no bf16 between
    float h[8];
    uint32_t am = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float gv = s[i >> 2][i & 3], uv = s[2 + (i >> 2)][i & 3];
      h[i] = gv / (1.0f + expf(-gv)) * uv;
      am = max(am, __float_as_uint(h[i]) & 0x7FFFFFFFu);
    }
    am = max(am, (uint32_t)__shfl_xor((int)am, 16));
    am = max(am, (uint32_t)__shfl_xor((int)am, 32));
    const bool nan = am >= 0x7F800000u;
    const uint32_t byte = nan ? 0xFFu : (uint32_t)max((int)(am >> 23) - 8, 0);
    const float mul = inv_scale_from_e8m0(nan ? 127u : byte);
    if (16 * c + l16 < m) {
      const int64_t item = s_item[16 * c + l16];
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        int q = cvt2_e4m3<false>(h[4 * b] * mul, h[4 * b + 1] * mul, 0);
        q = cvt2_e4m3<true>(h[4 * b + 2] * mul, h[4 * b + 3] * mul, q);
        *(int*)(a.h + item * N + n0 + 16 * b + 4 * g) = nan ? 0x7F7F7F7F : q;
      }
      if (g == 0) a.hs[item * (N / 32) + (n0 >> 5)] = (uint8_t)byte;
    }
  }
}

// ---------------------------------------------------------------------------
// Down projection and the weighted sum over a token's experts.  Columns of the
// matrix tile are tokens; a token that an expert does not have keeps its sum
// (a select, not a multiplication by zero, so that another token's expert with
// NaN weights does not reach it).
// ---------------------------------------------------------------------------
template <int WF, int CT>
__global__ __launch_bounds__(kMoeThreads) void moe_down_kernel(MoeArgs a) {
  __shared__ int s_ids[kMoeItems];
  __shared__ uint32_t s_bits[kMaxExperts / 32];
  __shared__ int s_hit[kMaxExperts];
  __shared__ v4f part[kMoeWaves][CT][64];
  load_ids(a, s_ids, s_bits);
  const int tid = threadIdx.x, lane = tid & 63, wv = uni(tid >> 6), l16 = lane & 15, g = lane >> 4;
  uint32_t word;
  int before;
  const int hit = count_hit(s_bits, word, before);
  if (wv == 0) {
    for (int i = before; word; ++i, word &= word - 1u) s_hit[i] = lane * 32 + __builtin_ctz(word);
  }
  if (a.status != nullptr && blockIdx.x == 0 && wv == 1) {
    bool bad = false;
    for (int i = lane; i < a.T * a.topk; i += 64) bad |= s_ids[i] < 0 || s_ids[i] >= a.E;
    const uint64_t any = __ballot(bad);
    if (lane == 0) a.status[0] = any != 0;
  }
  __syncthreads();
  const int64_t K = a.K, N = a.N, k0 = (int64_t)blockIdx.x * 16;
  const int64_t ldw = WF == kFmtE2M1 ? N / 2 : N;
  const int nch = (int)(N / 128), units = hit * nch, per = (units + kMoeWaves - 1) / kMoeWaves;
  v4f tot[CT], acc[CT];
  const uint8_t* hrow[CT];
  const uint8_t* hsrow[CT];
  bool have[CT], any[CT];
  float comb[CT];
#pragma unroll
  for (int c = 0; c < CT; ++c) {
    tot[c] = acc[c] = (v4f){0.f, 0.f, 0.f, 0.f};
    have[c] = any[c] = false;
    comb[c] = 0.f;
    hrow[c] = a.h;
    hsrow[c] = a.hs;
  }
  const uint8_t *wrow = a.q2, *srow = a.s2;
  auto flush = [&]() {
#pragma unroll
    for (int c = 0; c < CT; ++c) {
      if (!any[c]) continue;
      if (have[c]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) tot[c][i] += comb[c] * acc[c][i];
      }
      acc[c] = (v4f){0.f, 0.f, 0.f, 0.f};
    }
  };
  int cur = -1;
  const int end = min((wv + 1) * per, units);
  for (int u = wv * per; u < end; ++u) {
    const int x = u / nch, ch = u - x * nch;
    if (x != cur) {
      flush();
      cur = x;
      const int e = uni(s_hit[x]);
      wrow = a.q2 + ((int64_t)e * K + k0 + l16) * ldw;
      srow = a.s2 + (int64_t)e * K * (N / 32) + (k0 + l16) * 4 + g;
#pragma unroll
      for (int c = 0; c < CT; ++c) {
        const int t = 16 * c + l16;
        int first = -1;
        comb[c] = 0.f;
        if (t < a.T) {
          for (int j = 0; j < a.topk; ++j) {
            if (s_ids[t * a.topk + j] != e) continue;
            if (first < 0) first = t * a.topk + j;
            comb[c] += a.combine[t * a.topk + j];
          }
        }
        have[c] = first >= 0;
        any[c] = __ballot(have[c]) != 0;
        hrow[c] = a.h + (int64_t)max(first, 0) * N;
        hsrow[c] = a.hs + (int64_t)max(first, 0) * (N / 32) + g;
      }
    }
    const v8i wq = load_weight<WF>(wrow, ch, g);
    const int ws = srow[(int64_t)ch * K * 4];
#pragma unroll
    for (int c = 0; c < CT; ++c) {
      if (!any[c]) continue;
      v8i hq = (v8i){0, 0, 0, 0, 0, 0, 0, 0};
      int hs = 127;
      if (have[c]) {
        const v4i p = *(const v4i*)(hrow[c] + ch * 128 + 16 * g), q = *(const v4i*)(hrow[c] + ch * 128 + 64 + 16 * g);
        hq = (v8i){p[0], p[1], p[2], p[3], q[0], q[1], q[2], q[3]};
        hs = hsrow[c][ch * 4];
      }
      acc[c] = mfma<WF>(wq, ws, hq, hs, acc[c]);
    }
  }
  flush();
#pragma unroll
  for (int c = 0; c < CT; ++c) part[wv][c][lane] = tot[c];
  __syncthreads();
  for (int c = wv; c < CT; c += kMoeWaves) {
    const int t = 16 * c + l16;
    if (t >= a.T) continue;
    v4f s = part[0][c][lane];
#pragma unroll
    for (int v = 1; v < kMoeWaves; ++v) s += part[v][c][lane];
    *(v2i*)(a.out + (int64_t)t * K + k0 + 4 * g) =
        (v2i){(int)pack_bf16x2_rne(s[0], s[1]), (int)pack_bf16x2_rne(s[2], s[3])};
  }
}

template <int WF, int CT>
static hipError_t launch_moe_ct(const MoeArgs& a, hipStream_t st) {
  const int64_t slots = std::min<int64_t>(a.E, (int64_t)a.T * a.topk);
  hipLaunchKernelGGL((moe_gate_up_kernel<WF, CT>), dim3((unsigned)(a.N / kMoeRows), (unsigned)slots), dim3(kMoeThreads),
                     0, st, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((moe_down_kernel<WF, CT>), dim3((unsigned)(a.K / 16)), dim3(kMoeThreads), 0, st, a);
  return hipGetLastError();
}

// CT: tiles of 16 tokens that the accumulators hold.
template <int WF>
static hipError_t launch_moe_wf(const MoeArgs& a, hipStream_t st) {
  if (a.T <= 16) return launch_moe_ct<WF, 1>(a, st);
  if (a.T <= 32) return launch_moe_ct<WF, 2>(a, st);
  if (a.T <= 64) return launch_moe_ct<WF, 4>(a, st);
  return launch_moe_ct<WF, 8>(a, st);
}

hipError_t launch_moe_few_tokens(const MoeArgs& a, hipStream_t st) {
  return a.w_fp4 ? launch_moe_wf<kFmtE2M1>(a, st) : launch_moe_wf<kFmtE4M3>(a, st);
}

}  // namespace mxk
