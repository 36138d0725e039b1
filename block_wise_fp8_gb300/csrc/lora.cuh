// lora.cuh -- what the two forms of the low-rank adapters' products share: the
// tiles of tokens of one adapter, and small conversions.
#pragma once
#include "common.cuh"
#include "ptx.cuh"
#include "quant_math.cuh"

namespace fp8bq {
namespace {

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// What BF16(v) = hi leaves of v; nothing of an infinite one, which would make
// inf - inf of it.
__device__ __forceinline__ float low_half(float v, float hi) {
  return isinf(hi) ? 0.0f : v - hi;
}

struct Tile {
  int a, start, count;  // adapter (L: no adapter), first sorted row, rows
};

// The idx-th tile of the segments (rows offsets[a] .. offsets[a+1]-1 of
// adapter a, cut into tiles of ROWS rows; with `rest`, the rows after the
// last segment as adapter L).  One warp; count 0 when there is no such tile.
// Bounds outside [0, M] are clamped.
template <int ROWS>
__device__ Tile find_tile(const int *offsets, int L, int M, int idx, bool rest) {
  const int lane = threadIdx.x & 31;
  const int segs = L + (rest ? 1 : 0);
  const int per = (segs + 31) / 32;
  auto bound = [&](int k) { return k > L ? M : min(max(__ldg(offsets + k), 0), M); };
  int n = 0;
  for (int i = 0; i < per; ++i) {
    const int k = lane * per + i;
    if (k < segs) n += (max(bound(k + 1) - bound(k), 0) + ROWS - 1) / ROWS;
  }
  int upto = n;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int v = __shfl_up_sync(0xFFFFFFFFu, upto, d);
    if (lane >= d) upto += v;
  }
  const uint32_t past = __ballot_sync(0xFFFFFFFFu, upto > idx);
  Tile t = {L, 0, 0};
  if (past == 0) return t;
  const int owner = __ffs(past) - 1;
  if (lane == owner) {
    int left = idx - (upto - n);
    for (int i = 0; i < per; ++i) {
      const int k = lane * per + i;
      if (k >= segs) break;
      const int s = bound(k), len = max(bound(k + 1) - s, 0);
      const int tiles = (len + ROWS - 1) / ROWS;
      if (left < tiles) {
        t = {k, s + left * ROWS, min(ROWS, len - left * ROWS)};
        break;
      }
      left -= tiles;
    }
  }
  t.a = __shfl_sync(0xFFFFFFFFu, t.a, owner);
  t.start = __shfl_sync(0xFFFFFFFFu, t.start, owner);
  t.count = __shfl_sync(0xFFFFFFFFu, t.count, owner);
  return t;
}

__device__ __forceinline__ int rank_of(const LoraArgs &p, int a) {
  if (a >= p.L) return 0;
  return p.ranks ? min(max(__ldg(p.ranks + a), 0), p.R) : p.R;
}

}  // namespace
}  // namespace fp8bq
