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
//   moe_gate_up_kernel  blocks of 32 gate and 32 up rows of the hit experts (one
//                       scale block of h), for 16 or 32 of their tokens;
//   moe_down_kernel     32 or 16 output columns per workgroup, all hit experts, all
//                       tokens; the sum over a token's experts stays in fp32
//                       on the CU, so nothing is added through memory and the
//                       order of additions is fixed.  K / 32 workgroups leave
//                       CUs idle below K = 8192: 2.6 TB/s at K = 5120, one token.
// Partial sums of several waves are added in wave order.  A wave keeps the next
// lines of its weights in flight while it multiplies one.
//
// Matrix operand layout (v_mfma_scale_f32_16x16x128_f8f6f4): lane l holds row
// l%16, group g = l/16: E2M1 elements 32g..32g+31 in 16 bytes, E4M3 the
// 16-byte pieces g and g+4; its scale byte is block g's; its accumulators are
// column l%16, rows 4g..4g+3 (as with v_mfma_f32_16x16x32_bf16, which takes 8
// elements a lane, the same ones of both operands).  Weights are the first
// operand (rows), tokens the second (columns).
#include <algorithm>
#include <type_traits>

#include "mx_device.h"
#include "mx_kernels.h"
#include "mx_quantize.h"

namespace mxk {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

constexpr int kMoeWaves = 8, kMoeThreads = kMoeWaves * 64;
constexpr int kMoeRows = 32;                       // rows of h per block: one scale block
constexpr int kMoeCols = 16;                       // tokens per matrix tile
constexpr int kFmtE4M3 = 0, kFmtE2M1 = 4;          // the instruction's operand formats
constexpr int kLds = 160 * 1024;                   // of a CU

__device__ __forceinline__ int uni(int v) { return __builtin_amdgcn_readfirstlane(v); }

// Inclusive sum over the lanes of a wave: within rows of 16, then their totals
// into the rows after them.
__device__ __forceinline__ int scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);      // row_shr:1, 2, 4, 8
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);      // row_bcast:15, rows 1 and 3
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);      // row_bcast:31, rows 2 and 3
  return v;
}

// Slot of token t that names expert e first, or -1: a token that names an
// expert twice is one row of that expert.
__device__ __forceinline__ int slot_of(const int* s_ids, int t, int topk, int e) {
  int found = -1;
#pragma unroll 4
  for (int j = topk - 1; j >= 0; --j)
    if (s_ids[t * topk + j] == e) found = j;
  return found;
}

// ids of the call in LDS, and how many tokens name each expert.  Ids outside
// [0, E) name none.  (Whole numbers are added: the order does not matter.)
__device__ __forceinline__ void load_ids(const MoeArgs& a, int* s_ids, int* s_count) {
  const int tid = threadIdx.x, n = a.T * a.topk;
  for (int i = tid; i < a.E; i += kMoeThreads) s_count[i] = 0;
  for (int i = tid; i < n; i += kMoeThreads) s_ids[i] = a.ids[i];
  __syncthreads();
  for (int i = tid; i < n; i += kMoeThreads) {
    const int e = s_ids[i], t = i / a.topk;
    if (e >= 0 && e < a.E && slot_of(s_ids, t, a.topk, e) == i - t * a.topk) atomicAdd(&s_count[e], 1);
  }
  __syncthreads();
}

// Tokens of expert e in ascending order, found by a whole wave: token t goes to
// put(position, t, first slot); returns how many.
template <class F>
__device__ __forceinline__ int tokens_of(const MoeArgs& a, const int* s_ids, int e, F&& put) {
  const int lane = threadIdx.x & 63;
  int m = 0;
  for (int t0 = 0; t0 < a.T; t0 += 64) {
    const int t = t0 + lane;
    const int j = t < a.T ? slot_of(s_ids, t, a.topk, e) : -1;
    const uint64_t mask = __ballot(j >= 0);
    if (j >= 0) put(m + __builtin_popcountll(mask & ((1ull << lane) - 1)), t, j);
    m += __builtin_popcountll(mask);
  }
  return m;
}

// Buffer descriptor of `bytes` bytes from `base`.  Reads past the end give 0
// and touch no memory: kPast is an offset past every end, for loads that a
// pipeline issues beyond its last step.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void* base, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes, 0x00020000);
}
constexpr int kPast = 0x7FFFFFF0;

// Weights are read a line (128 bytes) of each row at a time, which is one
// 128-element chunk of E4M3 or two of E2M1: read by 64-byte halves, with other
// loads between, E2M1 lines came from memory twice and the layer ran at half
// the bandwidth.  A lane's two 16-byte pieces of a line are its operand of the
// chunk (E4M3), or those of the two chunks (E2M1).
template <int WF>
constexpr int kUnit = WF == kFmtE2M1 ? 2 : 1;      // chunks of a line

struct Weight {
  v4i p[2];
};

// The line at the descriptor's start of the weight row at byte offset `row`.
__device__ __forceinline__ Weight load_weight(__amdgpu_buffer_rsrc_t r, int row, int g) {
  const int o = row + 16 * g;
  return {{__builtin_amdgcn_raw_buffer_load_b128(r, o, 0, 0),
           __builtin_amdgcn_raw_buffer_load_b128(r, o + 64, 0, 0)}};
}

// Chunk `i` of a line as the instruction's first operand.
template <int WF>
__device__ __forceinline__ v8i operand(const Weight& w, int i) {
  if (WF == kFmtE2M1) return __builtin_shufflevector(w.p[i], w.p[i], 0, 1, 2, 3, -1, -1, -1, -1);
  return __builtin_shufflevector(w.p[0], w.p[1], 0, 1, 2, 3, 4, 5, 6, 7);
}

template <int M, int N, class F>
__device__ __forceinline__ void static_for(F&& f) {
  if constexpr (M < N) {
    f(std::integral_constant<int, M>{});
    static_for<M + 1, N>(f);
  }
}

template <int WF>
__device__ __forceinline__ v4f mfma(const v8i& w, int ws, const v8i& x, int xs, const v4f& c) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, c, WF, kFmtE4M3, 0, ws, 0, xs);
}

// The lane's 32 elements of a chunk as bf16 values, four operands of eight for
// the bf16 instruction.  Exact: E4M3 and E2M1 values times a power of two are
// bf16 numbers (NaN at scale byte 255; elements the library's quantizers made
// of bf16 values stay in range).
__device__ __forceinline__ void put_pair(v8bf& o, int at, bf16x2_t v) {
  o[at] = v[0];
  o[at + 1] = v[1];
}
// E4M3: two 16-byte pieces, each of one block.
__device__ __forceinline__ void to_bf16(const v4i p[2], float scale0, float scale1, v8bf out[4]) {
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float scale = i == 0 ? scale0 : scale1;
      v8bf& o = out[2 * i + j / 2];
      put_pair(o, 4 * (j & 1), __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)p[i][j], scale, false));
      put_pair(o, 4 * (j & 1) + 2, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)p[i][j], scale, true));
    }
}
// E2M1: one 16-byte piece of one block.
__device__ __forceinline__ void to_bf16(const v4i& p, float scale, v8bf out[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    put_pair(out[i], 0, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4((uint32_t)p[i], scale, 0));
    put_pair(out[i], 2, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4((uint32_t)p[i], scale, 1));
    put_pair(out[i], 4, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4((uint32_t)p[i], scale, 2));
    put_pair(out[i], 6, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4((uint32_t)p[i], scale, 3));
  }
}
// 2^(byte - 127) of byte `i` of four, for the converts (byte 0: as they read it).
__device__ __forceinline__ float scale_of(uint32_t bytes, int i) {
  return __uint_as_float((bytes >> (8 * i) & 0xFFu) << 23);
}

// First of the wave's `n` units; shares differ by one unit at most.
__device__ __forceinline__ int share(int n, int wv) { return (int)((int64_t)n * wv / kMoeWaves); }

// Workgroup barrier that orders LDS accesses and leaves loads from memory in
// flight (__syncthreads() would wait for them).
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// A dword per row in the lanes' four groups of 16 (a, b, c, d) -> lo: a and b
// each in all four groups, hi: c and d.
struct Spread {
  uint32_t lo[2], hi[2];
};
__device__ __forceinline__ Spread spread_rows(uint32_t v) {
  const auto h = __builtin_amdgcn_permlane32_swap(v, v, false, false);      // [a b a b], [c d c d]
  const auto l = __builtin_amdgcn_permlane16_swap(h[0], h[0], false, false);
  const auto u = __builtin_amdgcn_permlane16_swap(h[1], h[1], false, false);
  return {{l[0], l[1]}, {u[0], u[1]}};
}

// x / (1 + 2^(-x log2 e)): the power by the hardware, with what the product
// -x log2 e rounds away put back (2^-22 of it otherwise lost at x = -40), and a
// reciprocal of one ulp; some 2^-22 of the value in all, over the whole range of
// x.  From 2^100 on the one is lost beside the power, which is taken with 2^-160:
// its reciprocal would be subnormal past 2^126, which the hardware makes zero, and
// silu(-88) is -5.3e-37.  Where the product itself overflows (x past 2.36e38) the
// power is 0 or so large that the result is, with nothing to put back.
__device__ __forceinline__ float silu(float x) {
  const float y = -x * 1.442695041f, t = fminf(y, 280.f);
  const float lo = fmaf(-x, 1.925963033e-8f, fmaf(-x, 1.442695041f, -t));
  const bool far = t > 100.f;
  float p = __builtin_amdgcn_exp2f(far ? t - 160.f : t);
  p = fmaf(p * (fabsf(y) < 280.f ? lo : 0.f), 0.6931471806f, p);
  return __builtin_ldexpf(x * __builtin_amdgcn_rcpf((far ? 0.f : 1.f) + p), far ? -160 : 0);
}

// x in LDS: 128 codes (eight 16-byte pieces) per token and chunk, and the four
// scale bytes in an array of their own.  Piece p of token i is at p ^ i % 8: the
// same piece of eight consecutive tokens covers all banks.
constexpr int kCodes = 128, kRec = kCodes + 4;
__device__ __forceinline__ int piece(int token, int p) { return 16 * (p ^ (token & 7)); }

// ---------------------------------------------------------------------------
// Gate and up projection, SwiGLU and the quantization of h.
//
// A work entry is one hit expert with up to `rows` of its tokens (as many as
// LDS holds x of, 16 CT at most); the work is all entries' 32-row blocks of h,
// in order, dealt to the workgroups in equal runs, and a run's lines of weights
// to its eight waves in equal runs again.  A wave so has whole blocks, which it
// finishes alone, and at most a part of one at each end; those meet in LDS once,
// at the end of the run.  (With every block split over the eight waves, 28 lines
// of E2M1 made shares of 3 and 4, and all waves waited at every block: 128
// tokens, top 8 of 32 experts, K 7168, N 2048: 393 us the layer, 351 with whole
// blocks, in the same state of the rest.)
//
// Loads from memory are waited for in the order of their issue, so the wave's
// stream of weights, D lines of each row ahead and across the blocks, has no
// load in it that is wanted sooner: x is in LDS by then, and the scales come
// with the weights, one dword per row and chunk.
//
// The products are bf16 ones here, of the exact values: the block-scaled
// instruction drops the low bits of small products beside large ones (1.5e-4 of
// the sum of magnitudes on tokens with outliers), which moved values of h to a
// neighbouring code, and with one or seven tokens the output's error from 0.0017
// to 0.0042 and 0.0027.  It cost 21.9 -> 23.1 us (1 token) and 127 -> 130 (7) when
// it came in.  The down projection keeps the block-scaled instruction: with it the
// output's error is that of its rounding to bf16 (those 0.0017).
// ---------------------------------------------------------------------------
constexpr int kMoeGrid = 256;      // workgroups of the gate kernel, one per CU
static_assert(kMoeGrid == 1 << 8, "shares are taken by shifts");
// Row tiles (gate and up) whose sums meet in LDS at a time: with two column tiles
// one, as LDS is x's (20 tokens of K = 7168 and not 18: 128 tokens, top 4, 8-bit,
// 323 us against 336), else two, with half the barriers.
template <int CT>
constexpr int kParts = CT == 1 ? 2 : 1;

// ONE: a single token, whose experts every wave finds in registers, without the
// lists in LDS and their barriers (by the cycle counter 5000 cycles of the
// kernel's 34000).
template <int WF, int CT, bool ONE, int D>
__global__ __launch_bounds__(kMoeThreads) __attribute__((amdgpu_waves_per_eu(2))) void moe_gate_up_kernel(MoeArgs a,
                                                                                                          int rows) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  __shared__ v4f part[kMoeWaves][kParts<CT>][64];
  __shared__ int s_item[kMoeMaxTokens], s_token[kMoeMaxTokens], s_expert, s_pass, s_total;
  constexpr int U = kUnit<WF>;
  constexpr bool F4 = WF == kFmtE2M1;
  const int tid = threadIdx.x, lane = tid & 63, wv = uni(tid >> 6), l16 = lane & 15, g = lane >> 4;
  const int64_t K = a.K, N = a.N;
  const int nch = (int)(K / 128), lines = (nch + U - 1) / U, all = (int)(N / kMoeRows);
  const int ldw = (int)(F4 ? K / 2 : K);
  // x in LDS, [chunk][token]: codes, scales
  uint32_t* rsc = (uint32_t*)(smem + nch * rows * kCodes);
  int* s_ids = (int*)(smem + nch * rows * kRec);
  int *s_count = s_ids + a.T * a.topk, *s_upto = s_count + a.E;
  if constexpr (!ONE) load_ids(a, s_ids, s_count);
  // Work entry `entry` for the workgroup, by wave 0: its expert, pass and tokens;
  // by the one that has the entry's first block, what the down kernel needs.
  auto enter = [&](int entry, bool first_block) __attribute__((always_inline)) {
    int e = -1, rank = 0, prev = 0;      // rank: hit experts before it
    for (int base = 0; e < 0; base += 64) {
      const int i = base + lane;
      const uint64_t own = __ballot(i < a.E && (s_upto[min(i, a.E - 1)] & 0xFFFF) > entry);
      const uint64_t hits = __ballot(i < a.E && s_count[min(i, a.E - 1)] > 0);
      const int first = own ? __builtin_ctzll(own) : 64;
      rank += __builtin_popcountll(own ? hits & ((1ull << first) - 1) : hits);
      if (own) e = base + first;
    }
    if (e > 0) prev = s_upto[e - 1];
    const int pass = entry - (prev & 0xFFFF), off = prev >> 16;
    const bool leave = first_block && pass == 0;
    const int m = tokens_of(a, s_ids, e, [&](int i, int t, int j) {
      s_token[i] = t;
      s_item[i] = t * a.topk + j;
      if (leave) {
        // the row of h, the token and its weight (the sum, where it names the
        // expert twice)
        float c = 0.f;
        for (int k = 0; k < a.topk; ++k)
          if (s_ids[t * a.topk + k] == e) c += a.combine[t * a.topk + k];
        a.list[off + i] = make_int2((t * a.topk + j) | t << 16, __float_as_int(c));
      }
    });
    if (lane == 0) {
      if (leave) a.meta[1 + rank] = e | m << 16;
      s_expert = e;
      s_pass = pass;
    }
  };
  const uint32_t wg = blockIdx.x;
  uint32_t total;
  int id = -1, rank = 0;      // ONE: slot `lane`'s expert, and its place among the hit ones
  bool first = false;         // the slot is the first that names it
  if constexpr (ONE) {
    id = lane < a.topk ? a.ids[lane] : -1;
    first = id >= 0 && id < a.E;
    for (int j = 0; j < a.topk; ++j) {
      const int other = __builtin_amdgcn_readlane(id, j);
      first &= j >= lane || other != id;
    }
    const uint64_t firsts = __ballot(first);
    for (int j = 0; j < a.topk; ++j) {
      const int other = __builtin_amdgcn_readlane(id, j);
      rank += (firsts >> j & 1) != 0 && other < id;
    }
    const int hit = __builtin_popcountll(firsts);
    total = (uint32_t)hit * all;
    if (wg == 0 && wv == 0) {
      // for the down kernel, as in `enter`
      if (first) {
        float c = 0.f;
        for (int k = 0; k < a.topk; ++k)
          if (a.ids[k] == id) c += a.combine[k];
        a.list[rank] = make_int2(lane, __float_as_int(c));
        a.meta[1 + rank] = id | 1 << 16;
      }
      if (lane == 0) a.meta[0] = hit;
    }
  } else {
    if (wv == 0) {
      // entries (low half) and tokens (high half) of the experts up to each one:
      // at most 4096 of both
      int before = 0, hit = 0;
      for (int base = 0; base < a.E; base += 64) {
        const int c = base + lane < a.E ? s_count[base + lane] : 0;
        const int v = before + scan((c + rows - 1) / rows | c << 16);
        if (base + lane < a.E) s_upto[base + lane] = v;
        before = __builtin_amdgcn_readlane(v, 63);
        hit += __builtin_popcountll(__ballot(c > 0));
      }
      if (lane == 0) {
        s_total = (before & 0xFFFF) * all;
        if (wg == 0) a.meta[0] = hit;
      }
    }
    __syncthreads();
    total = (uint32_t)uni(s_total);
  }
  const int start = (int)((uint64_t)total * wg >> 8), stop = (int)((uint64_t)total * (wg + 1) >> 8);
  for (int at = start; at < stop;) {
    const int entry = at / all, b0 = at - entry * all, nb = min(all - b0, stop - at);
    if (at > start) __syncthreads();      // the lists and x of the entry before
    int e, m0 = 0, mp = 1, item_of_one = 0;
    if constexpr (ONE) {
      item_of_one = __builtin_ctzll(__ballot(first && rank == entry));
      e = __builtin_amdgcn_readlane(id, item_of_one);
    } else {
      if (wv == 0) enter(entry, b0 == 0);
      __syncthreads();
      e = uni(s_expert);
      // an expert's entries share its tokens evenly: a second column tile only
      // where the first one is full
      const int me = uni(s_count[e]), passes = (me + rows - 1) / rows, per = (me + passes - 1) / passes;
      m0 = uni(s_pass) * per;
      mp = min(me - m0, per);
    }
    at += nb;
    const bool wide = CT > 1 && mp > kMoeCols;        // a second column tile has tokens
    // the wave's lines, and the first one's block and place in it
    const int begin = share(nb * lines, wv), end = share(nb * lines, wv + 1);
    int b = begin / lines, u = begin - b * lines;

    // x: 16 lanes take 128 elements of a token; four loads, 16 of them, at a
    // time; a wave quantizes its share of the chunks
    const int q_begin = share(nch, wv) * mp, q_end = share(nch, wv + 1) * mp;
    // q / mp: q < 2^11 (LDS holds no more), so q * (2^17 / mp rounded up) is exact enough
    const uint32_t inv = ((1u << 17) + mp - 1) / mp;
    static_assert(kLds / kRec < 1 << 11 && (1 << 11) * 2 * kMoeCols < 1 << 17, "");
    v4i xw[4];
    auto load_x = [&](int q0) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int q = max(min(q0 + 4 * i + g, q_end - 1), 0), ch = (int)(q * inv >> 17), row = q - ch * mp;
        xw[i] = *(const v4i*)(a.x + (int64_t)(ONE ? 0 : s_token[m0 + row]) * K + ch * 128 + 8 * l16);
      }
    };
    auto store_x = [&](int q0) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int q = q0 + 4 * i + g;
        const us2 top = absmax8x2(xw[i]);
        const uint32_t byte = e8m0_from_absbits(quad_max(max(top[0], top[1])));
        const v2i c = quantize8(xw[i], byte, ((byte + 8u) << 7 | 0x60u) * 0x10001u);
        if (q < q_end) {
          const int row = q - (int)(q * inv >> 17) * mp;
          *(v2i*)(smem + q * kCodes + piece(row, l16 >> 1) + 8 * (l16 & 1)) =
              byte == 0xFFu ? (v2i){0x7F7F7F7F, 0x7F7F7F7F} : c;
          if ((l16 & 3) == 0) ((uint8_t*)(rsc + q))[l16 >> 2] = (uint8_t)byte;
        }
      }
    };
    // Four row tiles (two of gate rows, two of up rows) of a block.
    v4f acc[CT][4], head[CT][4];
    auto clear = [&](v4f (&t)[CT][4]) __attribute__((always_inline)) {
#pragma unroll
      for (int c = 0; c < CT; ++c)
#pragma unroll
        for (int r = 0; r < 4; ++r) t[c][r] = (v4f){0.f, 0.f, 0.f, 0.f};
    };
    clear(acc);
    clear(head);
    float h[8];
    uint32_t am;
    auto swiglu = [&](int r, const v4f& gs, const v4f& us) __attribute__((always_inline)) {
      if (r == 0) am = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        h[4 * r + i] = silu(gs[i]) * us[i];
        am = max(am, __float_as_uint(h[4 * r + i]) & 0x7FFFFFFFu);
      }
    };
    auto store_h = [&](int b, int c) __attribute__((always_inline)) {
      // rows 4g..4g+3 and 16 + 4g..; quantized from fp32, with no bf16 between
      am = max(am, (uint32_t)__shfl_xor((int)am, 16));
      am = max(am, (uint32_t)__shfl_xor((int)am, 32));
      const bool nan = am >= 0x7F800000u;
      const uint32_t byte = nan ? 0xFFu : (uint32_t)max((int)(am >> 23) - 8, 0);
      const float mul = inv_scale_from_e8m0(nan ? 127u : byte);
      const int token = kMoeCols * c + l16;
      if (token < mp) {
        const int64_t item = ONE ? item_of_one : s_item[m0 + token];
        const int n0 = (b0 + b) * kMoeRows;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          int q = cvt2_e4m3<false>(h[4 * r] * mul, h[4 * r + 1] * mul, 0);
          q = cvt2_e4m3<true>(h[4 * r + 2] * mul, h[4 * r + 3] * mul, q);
          *(int*)(a.h + item * N + n0 + 16 * r + 4 * g) = nan ? 0x7F7F7F7F : q;
        }
        if (g == 0) a.hs[item * (N / 32) + (n0 >> 5)] = (uint8_t)byte;
      }
    };
    // Block `b` was wholly this wave's.
    auto finish = [&](int b) __attribute__((always_inline)) {
#pragma unroll
      for (int c = 0; c < CT; ++c) {
        if (c > 0 && !wide) continue;
        swiglu(0, acc[c][0], acc[c][2]);
        swiglu(1, acc[c][1], acc[c][3]);
        store_h(b, c);
      }
    };

    Weight wq[D][4];
    uint32_t ws[D][U];
    // The next line to load: its place in the block, the first gate row there, how
    // far the block's rows reach from it; the scales of this lane's row, gate row l
    // or up row l - 32.
    int lu = u, reach = kMoeRows * ldw - u * 128;
    const int64_t to_up = N * ldw;
    const uint8_t* wp = a.q13 + (int64_t)e * 2 * to_up + (int64_t)(b0 + b) * (kMoeRows * ldw) + u * 128;
    const int64_t chunk = 2 * N * 4;      // bytes of a chunk's scales
    const uint8_t* sblock = a.s13 + e * (chunk * nch) + ((int64_t)(b0 + b) * kMoeRows + (lane < 32 ? lane : N + lane - 32)) * 4;
    const uint8_t* sp = sblock + u * U * chunk;
    const int row0 = l16 * ldw, row1 = row0 + 16 * ldw;
    auto load_w = [&](auto slot_c, bool live) __attribute__((always_inline)) {
      constexpr int S = decltype(slot_c)::value;
      const __amdgpu_buffer_rsrc_t rg = rsrc(wp, live ? reach : 0), ru = rsrc(wp + to_up, live ? reach : 0);
#pragma unroll
      for (int r = 0; r < 4; ++r) wq[S][r] = load_weight(r < 2 ? rg : ru, r & 1 ? row1 : row0, g);
      if (!live) return;
#pragma unroll
      for (int i = 0; i < U; ++i)      // an odd last chunk has no second one
        ws[S][i] = *(const uint32_t*)(sp + (i > 0 && lu * U + i < nch ? chunk : 0));
      wp += 128;
      reach -= 128;
      sp += U * chunk;
      if (++lu == lines) {
        lu = 0;
        wp += kMoeRows * ldw - lines * 128;
        reach = kMoeRows * ldw;
        sblock += kMoeRows * 4;
        sp = sblock;
      }
    };
    load_x(q_begin);       // ahead of the weights, which then load while it is quantized
    static_for<0, D>([&](auto sc) { load_w(sc, begin + decltype(sc)::value < end); });
    store_x(q_begin);
    for (int q0 = q_begin + 16; q0 < q_end; q0 += 16) {
      load_x(q0);
      store_x(q0);
    }
    lds_barrier();
    bool whole = u == 0;       // this wave has the block's first line
    for (int u0 = begin; u0 < end; u0 += D) {
      static_for<0, D>([&](auto sc) __attribute__((always_inline)) {
        constexpr int S = decltype(sc)::value;
        if (u0 + S < end) {
#pragma unroll
          for (int i = 0; i < U; ++i) {
            // an odd last chunk has no second one: its record is read again, its products dropped
            const int ch = min(u * U + i, nch - 1);
            const Spread sc4 = spread_rows(ws[S][i]);
            const uint32_t rs[4] = {sc4.lo[0], sc4.lo[1], sc4.hi[0], sc4.hi[1]};
            // elements 32g.. of E2M1, one block; pieces g and g+4 of E4M3, of
            // blocks g/2 and 2 + g/2
            const int s0 = F4 ? g : g >> 1, s1 = F4 ? g : 2 + (g >> 1);
            v8bf x4[CT][4];
#pragma unroll
            for (int c = 0; c < CT; ++c) {
              if (c > 0 && !wide) continue;
              const int token = min(kMoeCols * c + l16, mp - 1), row = ch * mp + token;
              const uint8_t* xr = smem + row * kCodes;
              const v4i xp[2] = {*(const v4i*)(xr + piece(token, F4 ? 2 * g : g)),
                                 *(const v4i*)(xr + piece(token, F4 ? 2 * g + 1 : 4 + g))};
              const uint32_t xs = rsc[row];
              to_bf16(xp, scale_of(xs, s0), scale_of(xs, s1), x4[c]);
            }
            if (u * U + i < nch) {
#pragma unroll
              for (int r = 0; r < 4; ++r) {
                v8bf w4[4];
                if constexpr (F4) to_bf16(wq[S][r].p[i], scale_of(rs[r], s0), w4);
                else to_bf16(wq[S][r].p, scale_of(rs[r], s0), scale_of(rs[r], s1), w4);
#pragma unroll
                for (int c = 0; c < CT; ++c) {
                  if (c > 0 && !wide) continue;
#pragma unroll
                  for (int j = 0; j < 4; ++j)
                    acc[c][r] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w4[j], x4[c][j], acc[c][r], 0, 0, 0);
                }
              }
            }
          }
          load_w(sc, u0 + S + D < end);
          if (++u == lines) {
            if (whole) {
              finish(b);
            } else {
#pragma unroll
              for (int c = 0; c < CT; ++c)
#pragma unroll
                for (int r = 0; r < 4; ++r) head[c][r] = acc[c][r];
            }
            clear(acc);
            whole = true;
            u = 0;
            ++b;
          }
        }
      });
    }
    // Blocks that several waves share: the first one (`whole`: it has the first
    // line) adds the others' sums, which are their heads, or all that they have.
    const bool shared = begin < end && u > 0;
    if (shared && !whole) {
#pragma unroll
      for (int c = 0; c < CT; ++c)
#pragma unroll
        for (int r = 0; r < 4; ++r) head[c][r] = acc[c][r];
    }
    if (nb % kMoeWaves != 0) {
#pragma unroll
      for (int c = 0; c < CT; ++c) {
        if (c > 0 && !wide) continue;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          v4f gu[2] = {acc[c][r], acc[c][2 + r]};
#pragma unroll
          for (int i = 0; i < 2; i += kParts<CT>) {
            lds_barrier();
#pragma unroll
            for (int k = 0; k < kParts<CT>; ++k) part[wv][k][lane] = head[c][2 * (i + k) + r];
            lds_barrier();
            if (shared && whole)
              for (int v = wv + 1; v < kMoeWaves && share(nb * lines, v) < (b + 1) * lines; ++v)
#pragma unroll
                for (int k = 0; k < kParts<CT>; ++k) gu[i + k] += part[v][k][lane];
          }
          if (shared && whole) {
            swiglu(r, gu[0], gu[1]);
            if (r == 1) store_h(b, c);
          }
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Down projection and the weighted sum over a token's experts.  A work entry
// is one hit expert with up to 16 CT of its tokens (columns of matrix tiles); the
// wave's share is a run of (entry, line) units, of which D are in registers or on
// their way, across the border between entries.  At the end of an entry its sums,
// times the combine weights, are added to the wave's own sums of those tokens in
// LDS.
// ---------------------------------------------------------------------------
template <int WF, int RT, int CT, int D>
__global__ __launch_bounds__(kMoeThreads) __attribute__((amdgpu_waves_per_eu(2))) void moe_down_kernel(MoeArgs a,
                                                                                                       int slots) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  __shared__ int s_entries;
  constexpr int U = kUnit<WF>, kCols = kMoeCols * CT;
  const int tid = threadIdx.x, lane = tid & 63, wv = uni(tid >> 6), l16 = lane & 15, g = lane >> 4;
  const int64_t K = a.K, N = a.N, k0 = (int64_t)blockIdx.x * 16 * RT;
  const int n = a.T * a.topk;
  // the waves' sums [T][16 RT], the tokens of all hit experts, the work entries
  // (expert | tokens << 16, and where they begin), what the gate kernel left
  v4f* sums = (v4f*)smem + (int64_t)wv * a.T * 4 * RT;
  int2* s_list = (int2*)(smem + (size_t)kMoeWaves * a.T * 64 * RT);
  int2* s_work = s_list + n;
  int* s_meta = (int*)(s_work + slots + n / kMoeCols);
  for (int i = tid; i < n; i += kMoeThreads) s_list[i] = a.list[i];      // past the hit experts' tokens: not used
  for (int i = tid; i <= slots; i += kMoeThreads) s_meta[i] = a.meta[i];
  for (int i = lane; i < a.T * 4 * RT; i += 64) sums[i] = (v4f){0.f, 0.f, 0.f, 0.f};
  __syncthreads();
  if (wv == 0) {
    const int hit = s_meta[0];
    int carry = 0, off = 0;
    for (int base = 0; base < hit; base += 64) {
      const int meta = base + lane < hit ? s_meta[1 + base + lane] : 0, m = meta >> 16;
      const int p = (m + kCols - 1) / kCols;
      const int incl = scan(p | m << 16);        // both running sums at once (at most 1280 entries, 4096 tokens)
      const int at = carry + (incl & 0xFFFF) - p, first = off + (incl >> 16) - m;
      for (int i = 0; i < p; ++i)
        s_work[at + i] = make_int2((meta & 0xFFFF) | min(m - i * kCols, kCols) << 16, first + i * kCols);
      const int last = __builtin_amdgcn_readlane(incl, 63);
      carry += last & 0xFFFF;
      off += last >> 16;
    }
    if (lane == 0) s_entries = carry;
  } else if (a.status != nullptr && blockIdx.x == 0 && wv == 1) {
    bool bad = false;
    for (int i = lane; i < n; i += 64) bad |= a.ids[i] < 0 || a.ids[i] >= a.E;
    const uint64_t any = __ballot(bad);
    if (lane == 0) a.status[0] = any != 0;
  }
  __syncthreads();
  const int ldw = (int)(WF == kFmtE2M1 ? N / 2 : N);
  const int entries = uni(s_entries);
  const int nch = (int)(N / 128), lines = (nch + U - 1) / U, units = entries * lines;
  const int begin = share(units, wv), end = share(units, wv + 1);
  const __amdgpu_buffer_rsrc_t rh = rsrc(a.h, (int64_t)n * N);
  const __amdgpu_buffer_rsrc_t rhs = rsrc(a.hs, (int64_t)n * (N / 32));
  if (begin < end) {
    // this lane's token in column tile c of a work entry: row of h | token << 16
    // (or -1), combine weight
    auto token_of = [&](int2 work, int c) __attribute__((always_inline)) {
      const int i = kMoeCols * c + l16;
      return i < work.x >> 16 ? s_list[work.y + i] : make_int2(-1, 0);
    };
    Weight wq[D][RT];
    v8i hq[D][CT][U];
    uint32_t ws[D];
    int hs[D][CT][U];
    int lx = begin / lines, lu = begin - lx * lines;      // entry and line of the next unit to load
    int item[CT];
    const uint8_t *wbase = nullptr, *sbase = nullptr;
    auto enter_load = [&]() __attribute__((always_inline)) {
      const int2 work = s_work[min(lx, entries - 1)];
      const int64_t e = uni(work.x & 0xFFFF);
#pragma unroll
      for (int c = 0; c < CT; ++c) {
        const int2 t = token_of(work, c);
        item[c] = t.x < 0 ? -1 : t.x & 0xFFFF;
      }
      wbase = a.q2 + (e * K + k0) * ldw;
      // scales: lane l's row is l % (16 RT), of the line's second chunk for l >= 32
      sbase = a.s2 + (e * K * (N / 128) + k0 + lane % (16 * RT)) * 4;
    };
    auto load = [&](auto slot_c, int u) __attribute__((always_inline)) {
      constexpr int S = decltype(slot_c)::value;
      const bool live = u < end;
      const __amdgpu_buffer_rsrc_t rw = rsrc(wbase + lu * 128, live ? (int64_t)16 * RT * ldw - lu * 128 : 0);
#pragma unroll
      for (int r = 0; r < RT; ++r) wq[S][r] = load_weight(rw, (16 * r + l16) * ldw, g);
      ws[S] = *(const uint32_t*)(sbase + (int64_t)min(lu * U + (U > 1 ? lane >> 5 : 0), nch - 1) * K * 4);
#pragma unroll
      for (int c = 0; c < CT; ++c)
#pragma unroll
        for (int i = 0; i < U; ++i) {
          const int ch = min(lu * U + i, nch - 1);       // a line's second chunk past the end is not used
          const bool have = live && item[c] >= 0;
          const int o = have ? item[c] * (int)N + ch * 128 + 16 * g : kPast - 64;
          const v4i p = __builtin_amdgcn_raw_buffer_load_b128(rh, o, 0, 0);
          const v4i q = __builtin_amdgcn_raw_buffer_load_b128(rh, o + 64, 0, 0);
          hq[S][c][i] = (v8i){p[0], p[1], p[2], p[3], q[0], q[1], q[2], q[3]};
          hs[S][c][i] =
              __builtin_amdgcn_raw_buffer_load_b8(rhs, have ? item[c] * (int)(N / 32) + ch * 4 + g : kPast, 0, 0);
        }
      if (++lu == lines) {
        lu = 0;
        ++lx;
        enter_load();
      }
    };
    v4f acc[CT][RT];
#pragma unroll
    for (int c = 0; c < CT; ++c)
#pragma unroll
      for (int r = 0; r < RT; ++r) acc[c][r] = (v4f){0.f, 0.f, 0.f, 0.f};
    int mx = lx, mu = lu;      // entry and line of the next unit to multiply
    auto flush = [&]() __attribute__((always_inline)) {
#pragma unroll
      for (int c = 0; c < CT; ++c) {
        const int2 mine = token_of(s_work[mx], c);
        const float w = __int_as_float(mine.y);
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          if (mine.x >= 0) {
            v4f* p = sums + ((mine.x >> 16) * RT + r) * 4 + g;
            v4f v = *p;
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] += w * acc[c][r][i];
            *p = v;
          }
          acc[c][r] = (v4f){0.f, 0.f, 0.f, 0.f};
        }
      }
    };
    enter_load();
    static_for<0, D>([&](auto sc) { load(sc, begin + decltype(sc)::value); });
    for (int u0 = begin; u0 < end; u0 += D) {
      static_for<0, D>([&](auto sc) __attribute__((always_inline)) {
        constexpr int S = decltype(sc)::value;
        if (u0 + S < end) {
          // row tiles r of chunk i: lo (i = 0) and hi (i = 1) hold theirs
          const Spread sp = spread_rows(ws[S]);
#pragma unroll
          for (int i = 0; i < U; ++i) {
            if (U > 1 && mu * U + i >= nch) continue;
#pragma unroll
            for (int r = 0; r < RT; ++r) {
              const uint32_t rs = i == 0 ? sp.lo[r] : sp.hi[r];
#pragma unroll
              for (int c = 0; c < CT; ++c)
                acc[c][r] =
                    mfma<WF>(operand<WF>(wq[S][r], i), (int)(rs >> (8 * g)), hq[S][c][i], hs[S][c][i], acc[c][r]);
            }
          }
          if (++mu == lines) {
            flush();
            mu = 0;
            ++mx;
          }
        }
        load(sc, u0 + S + D);
      });
    }
    if (mu > 0) flush();
  }
  __syncthreads();
  for (int i = tid; i < a.T * 4 * RT; i += kMoeThreads) {
    v4f s = ((const v4f*)smem)[i];
#pragma unroll
    for (int v = 1; v < kMoeWaves; ++v) s += ((const v4f*)smem)[(int64_t)v * a.T * 4 * RT + i];
    *(v2i*)(a.out + (int64_t)(i / (4 * RT)) * K + k0 + 4 * (i % (4 * RT))) =
        (v2i){(int)pack_bf16x2_rne(s[0], s[1]), (int)pack_bf16x2_rne(s[2], s[3])};
  }
}

// The most dynamic LDS a launch of the kernels may ask for, beside their static
// arrays: a kernel's limit is the process's, so it is the same in every call.
template <int CT>
constexpr int kGateLds = kLds - kMoeWaves * kParts<CT> * 1024 - kMoeMaxTokens * 8 - 256;
constexpr int kDownLds = kLds - 64;

template <int WF, int RT, int CT, bool ONE = false>
static hipError_t launch_moe(const MoeArgs& a, size_t down, hipStream_t st) {
  constexpr int DU = 2, DD = 2;
  const int64_t n = (int64_t)a.T * a.topk, slots = std::min<int64_t>(a.E, n);
  // x of as many tokens as LDS holds beside the partial sums and the lists
  const int64_t per_row = a.K / 128 * kRec, lists = (n + 2 * a.E) * 4;
  const int64_t fit = (kGateLds<CT> - lists) / per_row;
  const int rows = (int)std::min<int64_t>(std::min(a.T, CT * kMoeCols), fit);
  const size_t up = (size_t)(rows * per_row + lists);
  hipError_t e = hipFuncSetAttribute((const void*)moe_gate_up_kernel<WF, CT, ONE, DU>,
                                     hipFuncAttributeMaxDynamicSharedMemorySize, kGateLds<CT>);
  if (e != hipSuccess) return e;
  e = hipFuncSetAttribute((const void*)moe_down_kernel<WF, RT, CT, DD>, hipFuncAttributeMaxDynamicSharedMemorySize,
                          kDownLds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((moe_gate_up_kernel<WF, CT, ONE, DU>), dim3(kMoeGrid), dim3(kMoeThreads), up, st, a, rows);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((moe_down_kernel<WF, RT, CT, DD>), dim3((unsigned)(a.K / (16 * RT))), dim3(kMoeThreads), down, st, a,
                     (int)slots);
  return hipGetLastError();
}

// LDS of the down kernel with `rt` column tiles per workgroup.
static size_t down_lds(const MoeArgs& a, int rt) {
  const size_t n = (size_t)a.T * a.topk, slots = std::min<size_t>(a.E, n);
  return (size_t)kMoeWaves * a.T * 64 * rt + n * 8 + (slots + n / kMoeCols) * 8 + (slots + 1) * 4;
}

// Row tiles of the down kernel: two (h is read half as often) where the waves'
// sums of all tokens leave LDS for the lists, else one.  Column tiles: two where
// an expert has more than 8 tokens on average, so that few experts' weights are
// read twice.  Both kernels, us in a trace (16 experts, K 5120, N 8192 for one
// token, else 32 experts, K 7168, N 2048):
//                           as chosen   one row tile   the other column tiles
//   1 token, top 1, 4-bit      23.5         25.8           -
//   1 token, top 1, 8-bit      33.8         35.5           -
//   7 tokens, top 8, 4-bit      147          162          156 (two)
//   32, top 8, 4-bit (8 avg)    153          175          162 (two)
//   128, top 4, 4-bit           212          256          227 (one)
//   128, top 8, 4-bit           313          393          344 (one)
//   128, top 4, 8-bit           314          359          387 (one)
hipError_t launch_moe_few_tokens(const MoeArgs& a, hipStream_t st) {
  const size_t two = down_lds(a, 2), one = down_lds(a, 1);
  const bool wide = (int64_t)a.T * a.topk > 8 * (int64_t)a.E;
  if (a.T == 1) return a.w_fp4 ? launch_moe<kFmtE2M1, 2, 1, true>(a, two, st) : launch_moe<kFmtE4M3, 2, 1, true>(a, two, st);
  if (two <= kDownLds) {
    if (a.w_fp4) return wide ? launch_moe<kFmtE2M1, 2, 2>(a, two, st) : launch_moe<kFmtE2M1, 2, 1>(a, two, st);
    return wide ? launch_moe<kFmtE4M3, 2, 2>(a, two, st) : launch_moe<kFmtE4M3, 2, 1>(a, two, st);
  }
  if (a.w_fp4) return wide ? launch_moe<kFmtE2M1, 1, 2>(a, one, st) : launch_moe<kFmtE2M1, 1, 1>(a, one, st);
  return wide ? launch_moe<kFmtE4M3, 1, 2>(a, one, st) : launch_moe<kFmtE4M3, 1, 1>(a, one, st);
}

}  // namespace mxk
