// Output tiles of a rows-grouped product, found on the device.
//
// Rows [offs[e-1], offs[e]) of X belong to expert e; a tile is up to BM of one
// expert's rows by BN output columns.  The offsets never cross to the host:
// the launch covers an upper bound of the tiles, every workgroup counts the
// experts' M-tiles itself and takes its own, and the surplus workgroups leave.
#pragma once

#include "mx_device.h"
#include "mx_kernels.h"

namespace mxk {
namespace rows {

constexpr int kBand = 8;         // column tiles per band of the order
constexpr int kGroup = 4;        // M-tiles of an expert taken together
constexpr int kXcdChunk = 32;    // most consecutive tiles dealt to one XCD at a time

struct Tile {
  int valid;
  int e;
  int64_t i0, i_end;   // rows of X: [i0, min(i0 + BM, i_end))
  int64_t j0;
};

__device__ __forceinline__ int uni32(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ int64_t uni64(int64_t v) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)(uint64_t)v);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)((uint64_t)v >> 32));
  return (int64_t)(((uint64_t)hi << 32) | lo);
}

// Buffer descriptor of `bytes` bytes from `base`: reads past the end give 0.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void* base, int64_t bytes) {
  const int n = bytes > 0x7FFFFFFF ? 0x7FFFFFFF : (bytes < 0 ? 0 : (int)bytes);
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, n, 0x00020000);
}

// Rows of expert e.  Malformed offsets are clamped to [0, I] and made
// non-decreasing, so they cannot address out of bounds.
__device__ __forceinline__ void group(const int* offs, int e, int64_t I, int64_t& st, int64_t& en) {
  st = e == 0 ? 0 : (int64_t)offs[e - 1];
  en = (int64_t)offs[e];
  st = min(max(st, (int64_t)0), I);
  en = min(max(en, st), I);
}

// Tile of workgroup b.  The order runs in bands of kBand column tiles, expert
// by expert inside a band, in groups of kGroup of an expert's M-tiles, column
// tile by column tile.  The hardware deals workgroups round-robin over the 8
// XCDs (b % 8); chunks of kXcdChunk consecutive tiles go to one XCD and
// successive chunks to successive XCDs, so that the 32 CUs of an XCD work on
// 4 x 8 tiles whose L2 serves 12 panels instead of 64, and each XCD gets a
// slice of every expert.  A launch with fewer tiles than 8 chunks deals evenly.
// 16384 x 8192 x 5120, MXFP8 x MXFP4, against chunks of 16 with all of an
// expert's M-tiles together: one expert 487 us against 503, 16 experts 615
// against 632 (chunks of 64: 490 and 643).
template <int BM, int BN, int THREADS>
__device__ __forceinline__ Tile find_tile(const int32_t* __restrict__ g_offs, int E, int64_t I, int64_t J,
                                          int* s_offs, int* s_pref, int* s_total) {
  Tile d{};
  const int tid = threadIdx.x, lane = tid & 63;
  for (int e = tid; e < E; e += THREADS) s_offs[e] = g_offs[e];
  __syncthreads();
  if (tid < 64) {
    int carry = 0;
    for (int base = 0; base < E; base += 64) {
      const int e = base + lane;
      int tiles = 0;
      if (e < E) {
        int64_t st, en;
        group(s_offs, e, I, st, en);
        tiles = (int)((en - st + BM - 1) / BM);
      }
      int incl = tiles;
#pragma unroll
      for (int k = 1; k < 64; k <<= 1) {
        const int v = __shfl_up(incl, k);
        if (lane >= k) incl += v;
      }
      if (e < E) s_pref[e] = carry + incl - tiles;    // M-tiles of the experts before e
      carry += __shfl(incl, 63);
    }
    if (tid == 0) *s_total = carry;
  }
  __syncthreads();
  const int64_t mtiles = *s_total, ntj = (J + BN - 1) / BN;
  const int64_t total = mtiles * ntj;
  const int64_t chunk = total >= 8 * kXcdChunk ? kXcdChunk : (total + 7) / 8;
  if (chunk == 0) return d;
  const int64_t i = (int64_t)blockIdx.x >> 3;
  const int64_t t = ((i / chunk) * 8 + (blockIdx.x & 7)) * chunk + i % chunk;
  if (t >= total) return d;
  const int64_t band = t / (mtiles * kBand);
  const int64_t within = t - band * mtiles * kBand;
  const int64_t width = min((int64_t)kBand, ntj - band * kBand);
  const int64_t mw = within / width;
  int lo = 0, hi = E - 1;       // the last expert with s_pref <= mw owns M-tile mw
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (s_pref[mid] <= mw) lo = mid; else hi = mid - 1;
  }
  const int64_t cnt = (lo + 1 < E ? (int64_t)s_pref[lo + 1] : mtiles) - s_pref[lo];
  const int64_t r = within - (int64_t)s_pref[lo] * width;
  const int64_t first = r / (kGroup * width) * kGroup, size = min((int64_t)kGroup, cnt - first);
  const int64_t in_group = r - first * width;
  int64_t st, en;
  group(s_offs, lo, I, st, en);
  d.valid = 1;
  d.e = lo;
  d.i0 = st + (first + in_group % size) * BM;
  d.i_end = en;
  d.j0 = (band * kBand + in_group / size) * BN;
  return d;
}

// Workgroups that cover every tile of any offsets: sum_e ceil(m_e / BM) is at
// most I / BM + E, and at most I (an M-tile holds a row).
template <int BM, int BN>
inline int64_t grid(int64_t I, int64_t J, int64_t E) {
  int64_t m = (I + BM - 1) / BM + E;
  if (m > I) m = I;
  const int64_t tiles = m * ((J + BN - 1) / BN);
  return ((tiles + kXcdChunk - 1) / kXcdChunk + 7) / 8 * 8 * kXcdChunk;
}

}  // namespace rows
}  // namespace mxk
