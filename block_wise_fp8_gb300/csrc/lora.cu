// lora.cu -- low-rank adapters of many requests beside a shared projection:
// the grouping of tokens by adapter, and
//   y[t] = BF16(base[t] + s_a * B_a (A_a x[t])),   a the adapter of token t,
// with A_a [R, K], B_a [N, R] in BF16 and only the first ranks[a] rows of A_a
// and columns of B_a in use.
//
// Two products, two launches.  The first (shrink) leaves t = A_a x in FP32,
// split over K so that few tokens still fill the GPU; the second (expand) adds
// the splits in a fixed order, multiplies by B_a and adds the base row.  The
// rank is so small that both are bound by their long operands (x once, base
// and y once, the adapters once a tile): the tensor instruction takes its
// operands straight from global memory in registers.  That needs no shared
// memory because the K index of a product may be permuted at will if both
// operands agree: a lane takes 16 contiguous values of a 64-wide K block and
// feeds them to four MMAs, so every load is 16 bytes and a quad of lanes reads
// 128 contiguous bytes of a row.  In the same way the columns of the second
// product are dealt out so that a lane ends with 8 neighbouring outputs.
//
// Measured with inputs changing from call to call: 6.2 us for one token and 10.2 us
// for 64 tokens of 32 adapters of mixed rank up to 32, 6144 -> 6144 (17 MB; 2.6 us
// at HBM's rate; with one input over and over 5.0 and 11.7).  What is left is
// latency: two kernels of one pass each, the way from offsets over order to the
// first row, and the splits' sums, read back by every column block.
//
// t enters the second product as the sum of two BF16 values (hi + lo, 16
// significant bits; the rounding left is 2^-17 of t, below the FP32 sums' own
// noise at these lengths and far below the output's 2^-9), so that y carries
// one BF16 rounding, its own.
#include "lora.cuh"

namespace fp8bq {
namespace {

// Tokens of one adapter that a CTA takes: two 16-row MMA tiles, the same for each
// of its warps, which share out K or the columns.  (Tiles of 128, a warp's own 32
// tokens each, left a warp all of K: 24.7 us for 44 tokens of one adapter of rank
// 56, 1200 -> 2648, against 11.7.)
constexpr int kTile = 32;
constexpr int kLoraThreads = 128;

// D (16x8, FP32) += A (16x16, BF16) B (16x8, BF16)
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// t = A_a x over one K split, 64 ranks at most (a higher rank takes a second
// plane of CTAs, which finds x in L2).  The K blocks are dealt to the four warps,
// whose sums are joined in a fixed order.
template <int NT>  // 8-row groups of A: min(R, 64) <= 8 NT
__global__ void __launch_bounds__(kLoraThreads) lora_shrink_kernel(const LoraArgs p) {
  __shared__ float red[3][NT * 8][32];
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int g = lane >> 2, q = lane & 3;
  const int M = static_cast<int>(p.M);
  const Tile t = find_tile<kTile>(p.offsets, p.L, M, blockIdx.x, false);
  const int r0 = blockIdx.z * (NT * 8);  // first rank of this plane
  const int rank = rank_of(p, t.a) - r0;
  if (t.count == 0 || rank <= 0) return;
  const bool two = t.count > 16;

  const uint16_t *xr[2][2];
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int row = m * 16 + r * 8 + g;
      xr[m][r] = nullptr;
      if (row < t.count) {
        const int tok = __ldg(p.order + t.start + row);
        if (tok >= 0 && tok < M) xr[m][r] = p.x + tok * p.ldx + 16 * q;
      }
    }
  const uint16_t *ar[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n)
    ar[n] = n * 8 + g < rank ? p.a + (static_cast<int64_t>(t.a) * p.R + r0 + n * 8 + g) * p.K + 16 * q
                             : nullptr;

  float acc[2][NT][4];
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[m][n][i] = 0.0f;

  const int kb0 = blockIdx.y * p.kb_split;
  const int kb1 = min((p.K + 63) / 64, kb0 + p.kb_split);
  const uint4 zero = make_uint4(0, 0, 0, 0);
  constexpr int kUnroll = NT <= 4 ? 2 : 1;
#pragma unroll kUnroll
  for (int kb = kb0 + w; kb < kb1; kb += 4) {
    const int k = kb * 64;
    const bool in = k + 16 * q < p.K;
    uint4 xv[2][2][2], av[NT][2];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const bool on = in && xr[m][r] != nullptr;
        const uint4 *src = reinterpret_cast<const uint4 *>(xr[m][r] + k);
        xv[m][r][0] = on ? __ldg(src) : zero;
        xv[m][r][1] = on ? __ldg(src + 1) : zero;
      }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const bool on = in && ar[n] != nullptr;
      const uint4 *src = reinterpret_cast<const uint4 *>(ar[n] + k);
      av[n][0] = on ? __ldg(src) : zero;
      av[n][1] = on ? __ldg(src + 1) : zero;
    }
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      if (m == 1 && !two) break;
      const uint32_t x0[8] = {xv[m][0][0].x, xv[m][0][0].y, xv[m][0][0].z, xv[m][0][0].w,
                              xv[m][0][1].x, xv[m][0][1].y, xv[m][0][1].z, xv[m][0][1].w};
      const uint32_t x1[8] = {xv[m][1][0].x, xv[m][1][0].y, xv[m][1][0].z, xv[m][1][0].w,
                              xv[m][1][1].x, xv[m][1][1].y, xv[m][1][1].z, xv[m][1][1].w};
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if (n * 8 >= rank) break;
        const uint32_t b[8] = {av[n][0].x, av[n][0].y, av[n][0].z, av[n][0].w,
                               av[n][1].x, av[n][1].y, av[n][1].z, av[n][1].w};
#pragma unroll
        for (int s = 0; s < 4; ++s)
          mma_bf16(acc[m][n], x0[2 * s], x1[2 * s], x0[2 * s + 1], x1[2 * s + 1], b[2 * s],
                   b[2 * s + 1]);
      }
    }
  }

  if (w > 0) {
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) red[w - 1][(m * NT + n) * 4 + i][lane] = acc[m][n][i];
  }
  __syncthreads();
  if (w > 0) return;
#pragma unroll
  for (int o = 0; o < 3; ++o)
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[m][n][i] += red[o][(m * NT + n) * 4 + i][lane];
  float *out = p.part + (static_cast<int64_t>(blockIdx.y) * p.M + t.start) * p.R;
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int row = m * 16 + r * 8 + g;
      if (row >= t.count) continue;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int c = r0 + n * 8 + 2 * q;
        if (c < p.R)
          *reinterpret_cast<float2 *>(out + static_cast<int64_t>(row) * p.R + c) =
              make_float2(acc[m][n][2 * r], acc[m][n][2 * r + 1]);
      }
    }
}

// y = base + s_a * B_a t.  The warps lay t out as MMA operands in shared memory,
// each a part of it, and walk the groups of 32 columns, each every fourth.  Rows
// without an adapter come as a tile of rank 0 and are copied.
template <int KS>  // 16-wide steps of the rank: R <= 16 KS
__global__ void __launch_bounds__(kLoraThreads) lora_expand_kernel(const LoraArgs p) {
  extern __shared__ uint4 sm[];
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int g = lane >> 2, q = lane & 3;
  const int M = static_cast<int>(p.M);
  // the first product's launch waited for everything before it, so what it
  // read (offsets, order, weights) and the base rows are visible here already
  const Tile t = find_tile<kTile>(p.offsets, p.L, M, blockIdx.x, p.copy_rest != 0);
  if (t.count == 0) {  // nothing to do, but this grid must not end before the first product's
    griddep_wait();
    return;
  }
  const bool two = t.count > 16;
  const int rank = rank_of(p, t.a);
  const int ks_n = (rank + 15) / 16;
  uint4 *my = sm + lane;  // [ks][m][hi, lo][lane]

  int tok[2][2];
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int row = m * 16 + r * 8 + g;
      const int v = row < t.count ? __ldg(p.order + t.start + row) : -1;
      tok[m][r] = v < M ? v : -1;
    }

  const int groups = (p.N + 31) / 32;
  const int g0 = blockIdx.y * p.ngroups;
  const int g1 = min(groups, g0 + p.ngroups);
  const uint4 zero = make_uint4(0, 0, 0, 0);
  const uint16_t *bw = p.b + static_cast<int64_t>(t.a) * p.N * p.R + 4 * q;
  // Column groups whose loads are in flight (64 tokens of 32 adapters, rank 32,
  // 6144 -> 6144: 13.0 us for both kernels with two, 13.5 with one, 15.2 with
  // three, which take too many registers, as two do at higher ranks)
  constexpr int kAhead = KS <= 2 ? 2 : 1;
  uint4 bsp[kAhead][2][2];
  uint2 bvp[kAhead][KS][4];
  // a column group's base and B: not t's, so the first groups' are asked for
  // while the first product still runs
  auto load = [&](int cg, uint4(&bs)[2][2], uint2(&bv)[KS][4]) {
    const int n0 = cg * 32, nc = n0 + 8 * q;
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int r = 0; r < 2; ++r)
        bs[m][r] = tok[m][r] >= 0 && nc < p.N
                       ? *reinterpret_cast<const uint4 *>(p.base + tok[m][r] * p.ldbase + nc)
                       : zero;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int col = n0 + (g >> 1) * 8 + 2 * j + (g & 1);
        const int k = ks * 16 + 4 * q;
        bv[ks][j] = make_uint2(0, 0);
        if (col < p.N && k < rank)
          bv[ks][j] = __ldg(reinterpret_cast<const uint2 *>(
              bw + static_cast<int64_t>(col) * p.R + ks * 16));
      }
  };
  constexpr int kStep = kLoraThreads / 32;
  const int first = g0 + w;
#pragma unroll
  for (int u = 0; u < kAhead; ++u)
    if (first + u * kStep < g1) load(first + u * kStep, bsp[u], bvp[u]);

  griddep_wait();
  if (rank > 0) {
    const float scale = __ldg(p.scales + t.a);
    const float *src = p.part + static_cast<int64_t>(t.start) * p.R;
    for (int i = w; i < ks_n * 2; i += kLoraThreads / 32) {
      const int ks = i >> 1, m = i & 1, k = ks * 16 + 4 * q;
      if (m == 1 && !two) continue;
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int row = m * 16 + r * 8 + g;
        float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (row < t.count && k < p.R) {
          const float *at = src + static_cast<int64_t>(row) * p.R + k;
#pragma unroll 8
          for (int s = 0; s < p.splits; ++s) {
            const float4 f = __ldcg(reinterpret_cast<const float4 *>(at + s * p.M * p.R));
            v[0] += f.x, v[1] += f.y, v[2] += f.z, v[3] += f.w;
          }
        }
        float l[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[i] = k + i < rank ? v[i] * scale : 0.0f;
          l[i] = low_half(v[i], __uint_as_float(pack_bf16(0.0f, v[i]) & 0xFFFF0000u));
        }
        hi[r] = pack_bf16(v[0], v[1]), hi[2 + r] = pack_bf16(v[2], v[3]);
        lo[r] = pack_bf16(l[0], l[1]), lo[2 + r] = pack_bf16(l[2], l[3]);
      }
      my[((ks * 2 + m) * 2 + 0) * 32] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      my[((ks * 2 + m) * 2 + 1) * 32] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
  }
  __syncthreads();

  auto product = [&](int cg, uint4(&bs)[2][2], uint2(&bv)[KS][4]) {
    const int nc = cg * 32 + 8 * q;  // this lane's 8 output columns
    if (rank & 15) {  // columns past the rank are not used as numbers
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        const int k = ks * 16 + 4 * q;
        if (k + 4 <= rank) continue;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (k + 3 >= rank) bv[ks][j].y &= 0xFFFFu;
          if (k + 2 >= rank) bv[ks][j].y = 0;
          if (k + 1 >= rank) bv[ks][j].x &= 0xFFFFu;
        }
      }
    }
    float acc[2][4][4];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[m][j][i] = 0.0f;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      if (ks >= ks_n) break;
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        if (m == 1 && !two) break;
        const uint4 hi = my[((ks * 2 + m) * 2 + 0) * 32];
        const uint4 lo = my[((ks * 2 + m) * 2 + 1) * 32];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          mma_bf16(acc[m][j], hi.x, hi.y, hi.z, hi.w, bv[ks][j].x, bv[ks][j].y);
          mma_bf16(acc[m][j], lo.x, lo.y, lo.z, lo.w, bv[ks][j].x, bv[ks][j].y);
        }
      }
    }
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        if (tok[m][r] < 0 || nc >= p.N) continue;
        const uint32_t bb[4] = {bs[m][r].x, bs[m][r].y, bs[m][r].z, bs[m][r].w};
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          o[j] = pack_bf16(bf16_lo(bb[j]) + acc[m][j][2 * r],
                           bf16_hi(bb[j]) + acc[m][j][2 * r + 1]);
        *reinterpret_cast<uint4 *>(p.y + tok[m][r] * p.ldy + nc) =
            make_uint4(o[0], o[1], o[2], o[3]);
      }
  };
#pragma unroll 1
  for (int cg = first; cg < g1; cg += kAhead * kStep)
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int at = cg + u * kStep;
      if (at >= g1) break;
      product(at, bsp[u], bvp[u]);
      if (at + kAhead * kStep < g1) load(at + kAhead * kStep, bsp[u], bvp[u]);
    }
}

// Stable counting sort of tokens by adapter in one cluster of C CTAs: each warp
// counts its own stretch of tokens in its own row of counters (the equal keys of
// 32 tokens are found with a ballot a bit and added by one lane: no atomics, so
// the order is fixed), the counters are scanned key by key, over the warps, then
// over the CTAs, and each warp writes its stretch.  The bytes are nothing; the
// barriers and a warp's walk over its tokens are what it takes.  Measured with
// one set of tokens in random order, over and over: 2.3 us for 64 tokens of 32 adapters, 6.3 us for 16384 of
// 128 (23 in one CTA; with a match of the lanes' keys, which goes through the
// different keys one by one, 9.5 and 48).  Up to 1024 tokens, 32 a warp, a
// cluster's start costs more than it saves: 3.5 us in one CTA, 4.3 in eight; from
// there on the eight win (2048 tokens: 4.6 and 4.35, 4096: 6.7 and 4.4).
constexpr int kGroupThreads = 1024;
constexpr int kGroupCluster = 8;
constexpr int kGroupOneCta = 1024;
__host__ __device__ constexpr int group_stretch(int M, int C) {  // tokens of a warp
  return ((M + 32 * C - 1) / (32 * C) + 31) / 32 * 32;
}

__device__ __forceinline__ int ld_cluster(uint32_t addr) {
  int v;
  asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

template <int C>
__global__ void __launch_bounds__(kGroupThreads) lora_group_kernel(const int *ids, int M, int L,
                                                                   int *order, int *offsets) {
  extern __shared__ int cnt[];  // [warps][L + 1]
  __shared__ int wsum[32];
  __shared__ int start[kMaxAdapters + 1];               // where this CTA's tokens of a key go
  __shared__ int of_cta[C > 1 ? kMaxAdapters + 1 : 1];  // how many they are
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int keys = L + 1;
  const int each = group_stretch(M, C);
  constexpr int kWarps = kGroupThreads / 32;
  const int warps = M ? min(kWarps, (M - 1) / each + 1) : 0;  // with tokens
  for (int i = threadIdx.x; i < warps * keys; i += kGroupThreads) cnt[i] = 0;
  __syncthreads();
  const int64_t from = (static_cast<int64_t>(blockIdx.x) * kWarps + w) * each;
  const int begin = static_cast<int>(from < M ? from : M);
  const int end = static_cast<int>(from + each < M ? from + each : M);
  int *mine = cnt + w * keys;
  auto walk = [&](auto &&at) {
    auto fetch = [&](int i) { return i < end ? __ldg(ids + i) : 0; };
    int id[4];  // this step's and the next three's
#pragma unroll
    for (int u = 0; u < 4; ++u) id[u] = fetch(begin + u * 32 + lane);
#pragma unroll 1
    for (int i0 = begin; i0 < end; i0 += 32) {
      const int i = i0 + lane, id0 = id[0];
      id[0] = id[1], id[1] = id[2], id[2] = id[3], id[3] = fetch(i + 128);
      // the lanes with this lane's key, a ballot a bit of it
      const int key = id0 >= 0 && id0 < L ? id0 : L;
      uint32_t same = __ballot_sync(0xFFFFFFFFu, i < end);
#pragma unroll
      for (int b = 0; b < 10; ++b) {
        if (L >> b == 0) break;
        const uint32_t ones = __ballot_sync(0xFFFFFFFFu, key >> b & 1);
        same &= key >> b & 1 ? ones : ~ones;
      }
      at(i, key, same);  // by all lanes
      __syncwarp();
    }
  };
  walk([&](int i, int key, uint32_t same) {
    if (i < end && (same & ((1u << lane) - 1u)) == 0) mine[key] += __popc(same);
  });
  __syncthreads();
  // exclusive positions: keys in order, a key's warps in order
  const int key = threadIdx.x;
  int total = 0;
  if (key < keys)
    for (int i0 = 0; i0 < warps; i0 += 8) {
      int c[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) c[i] = i0 + i < warps ? cnt[(i0 + i) * keys + key] : 0;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i0 + i < warps) {
          cnt[(i0 + i) * keys + key] = total;
          total += c[i];
        }
    }
  int before = 0;  // this key's tokens in the CTAs before this one
  if constexpr (C > 1) {
    if (key < keys) of_cta[key] = total;
    __syncwarp();
    cluster_sync();
    total = 0;
    if (key < keys) {
      int n[C];
#pragma unroll
      for (int c = 0; c < C; ++c) n[c] = ld_cluster(mapa_shared(smem_u32(&of_cta[key]), c));
#pragma unroll
      for (int c = 0; c < C; ++c) {
        if (c == static_cast<int>(blockIdx.x)) before = total;
        total += n[c];
      }
    }
  }
  int upto = total;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int v = __shfl_up_sync(0xFFFFFFFFu, upto, d);
    if (lane >= d) upto += v;
  }
  if (lane == 31) wsum[w] = upto;
  __syncthreads();
  if (w == 0) {
    int v = wsum[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xFFFFFFFFu, v, d);
      if (lane >= d) v += o;
    }
    wsum[lane] = v;
  }
  __syncthreads();
  const int base = upto - total + (w ? wsum[w - 1] : 0);
  if (key < keys) {
    if (blockIdx.x == 0) offsets[key] = base;
    start[key] = base + before;
  }
  __syncthreads();
  walk([&](int i, int key_i, uint32_t same) {
    const int rank = __popc(same & ((1u << lane) - 1u));
    const int at = start[key_i] + mine[key_i] + rank;
    __syncwarp();  // every lane has read its counter
    if (i < end) {
      order[at] = i;
      if (rank == 0) mine[key_i] += __popc(same);
    }
  });
  __syncwarp();
  if constexpr (C > 1) cluster_sync();  // no CTA leaves while another reads its counts
}

}  // namespace

// Which form runs.  The form for many tokens has HBM's rate but costs about 15 us
// before it does anything, and it moves 128 tokens of an adapter at a time; the
// direct form's time goes with the products, M R (K + N).  So the former runs from
// a certain size of these on, and where its tiles are full enough for the rank (in
// the direct form a higher rank costs more for the same bytes).  Measured, direct
// and other, us:  M 1024, 4 adapters, rank 64, 4096 -> 14336 (M R (K + N) = 1.2e9)
// 31 and 34, M 2048 52 and 42; M 2048, rank 32, 6144 -> 6144 (0.8e9) 27 and 28, M
// 4096 43 and 40; M 4096, 16 adapters, rank 64, 6144 -> 24576 153 and 107, 32 of
// them 165 and 141; M 2048 of 32 104 and 98, of 64 130 and 176; rank 32, 2048 ->
// 12288, M 8192, 16 adapters 97 and 90, 32 of them 100 and 114; rank 128, 4096 ->
// 4096, M 2048, 32 adapters 60 and 49, M 1536 of 64 59 and 79.  L is the table's
// size, all that the host knows, and stands for the adapters of the batch: 4096
// tokens of four adapters, rank 64, 6144 -> 24576, take 96 us with a table of up
// to 32, 188 in one of 64, where the direct form runs, and 236 in one of 128.
bool lora_is_large(int64_t M, int64_t N, int64_t K, int64_t L, int64_t R) {
  return M >= kLoraLargeTokens && M * R >= 1300000000 / (K + N) && M * R * R >= 320 * 1024 * L &&
         M >= 32 * L;
}

// Splits of the first product.  Direct form: enough that each warp has a K block
// (four a split) up to 8 tokens, fewer above, where there are more tiles and the
// second product reads every split's sums for every column group.  Many tokens: a
// CTA an SM over about M / 128 + 2 tiles.
int lora_splits(int64_t M, int64_t K, bool large, int *kb_split) {
  const int kbs = static_cast<int>((K + 63) / 64);
  int splits = !large ? (M <= 8 ? 24 : 8) : static_cast<int>(152 / (M / 128 + 2));
  if (splits > 24) splits = 24;
  if (splits > (kbs + 3) / 4) splits = (kbs + 3) / 4;
  if (splits < 1) splits = 1;
  const int per = (kbs + splits - 1) / splits;
  *kb_split = per;
  return (kbs + per - 1) / per;
}

cudaError_t launch_lora_add(LoraArgs a, int num_sms, cudaStream_t st) {
  const bool large = lora_is_large(a.M, a.N, a.K, a.L, a.R);
  a.splits = lora_splits(a.M, a.K, large, &a.kb_split);
  a.copy_rest = a.y != a.base;
  if (large) return launch_lora_large(a, num_sms, st);
  // each segment adds at most one partly filled tile; none is empty
  const int64_t full = (a.M + kTile - 1) / kTile;
  const int64_t shrink_tiles = full + a.L < a.M ? full + a.L : a.M;
  const int64_t expand_tiles = full + a.L + 1 < a.M ? full + a.L + 1 : a.M;
  {
    const dim3 grid(static_cast<unsigned>(shrink_tiles), a.splits), block(kLoraThreads);
    cudaError_t e;
    if (a.R <= 16) e = launch_pdl(lora_shrink_kernel<2>, grid, block, 0, st, a);
    else if (a.R <= 32) e = launch_pdl(lora_shrink_kernel<4>, grid, block, 0, st, a);
    else e = launch_pdl(lora_shrink_kernel<8>, dim3(grid.x, grid.y, (a.R + 63) / 64), block, 0, st, a);
    if (e != cudaSuccess) return e;
  }
  const int groups = (a.N + 31) / 32;
  int64_t ng = (groups * expand_tiles + num_sms * 4 - 1) / (num_sms * 4);
  ng = (ng + 3) / 4 * 4;
  a.ngroups = static_cast<int>(ng < groups ? ng : groups);
  const dim3 grid(static_cast<unsigned>(expand_tiles), (groups + a.ngroups - 1) / a.ngroups),
      block(kLoraThreads);
  const int ks = (a.R + 15) / 16;
  auto expand = [&](auto k) {
    constexpr int KS = decltype(k)::value;
    constexpr int smem = KS * 2 * 2 * 32 * 16;
    return launch_pdl(lora_expand_kernel<KS>, grid, block, smem, st, a);
  };
  if (ks <= 1) return expand(std::integral_constant<int, 1>{});
  if (ks <= 2) return expand(std::integral_constant<int, 2>{});
  if (ks <= 4) return expand(std::integral_constant<int, 4>{});
  return expand(std::integral_constant<int, 8>{});
}

cudaError_t launch_lora_group(const int *ids, int64_t M, int L, int *order, int *offsets,
                              cudaStream_t st) {
  const size_t smem = static_cast<size_t>(kGroupThreads / 32) * (L + 1) * sizeof(int);
  auto run = [&](auto c) {
    constexpr int C = decltype(c)::value;
    // (always: the default limit of 48 KB counts the static arrays too)
    cudaError_t e = allow_smem<lora_group_kernel<C>>(kGroupThreads / 32 * (kMaxAdapters + 1) *
                                                     sizeof(int));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {C, 1, 1};
    cfg.gridDim = dim3(C);
    cfg.blockDim = dim3(kGroupThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, lora_group_kernel<C>, ids, static_cast<int>(M), L, order,
                              offsets);
  };
  return M > kGroupOneCta ? run(std::integral_constant<int, kGroupCluster>{})
                          : run(std::integral_constant<int, 1>{});
}

}  // namespace fp8bq
