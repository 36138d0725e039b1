// lora_large.cu -- the low-rank adapters' two products for many tokens (lora.cu
// has the formulas and the form for few), on tcgen05 with TMEM accumulators.
//
// Both are bound by HBM: the first reads x once, the second reads base and
// writes y once, and the rank is too small to keep the tensor cores busy.  What
// carries them is bytes in flight, all of it asynchronous:
//
//   shrink  a CTA takes 128 tokens and one of the K splits.  Eight warps copy the
//           tokens' rows (in the order's order) and A_a's rows into a ring of
//           128-byte-swizzled stages with cp.async, one thread issues the MMAs
//           (128 tokens x rank, K = 64 a stage).
//           The last split of a tile to finish adds them up and writes t as the
//           second product's operand, so that no CTA of that one adds again.
//   expand  persistent CTAs take equal runs of (128 tokens, 128 columns) blocks.
//           Two groups of four warps have a token a thread: base comes into
//           shared memory by TMA, a block of the group's ahead, the product's row
//           is added to it from TMEM in place, and TMA takes it to y.  B_a's rows
//           come by cp.async; what lies past the adapter's rank is not read but
//           filled with zeros by the copy.
//
// The direct form reads operands straight into registers, which leaves little in
// flight: 146 us at 4096 tokens, 6144 -> 24576, rank 64, where these take 17 + 62
// us (x at 3.0 TB/s: 32 tiles of tokens in a few splits are too few bytes in
// flight for more; base and y at 6.6 TB/s, HBM's rate) and 94 us with the two
// launches and the hand-over of t between them.
#include "lora.cuh"

namespace fp8bq {
namespace {

// Instruction descriptor, kind::f16: D = F32 (bits 4-5 = 1), A and B BF16 (bits
// 7-9, 10-12 = 1), both K-major, N >> 3 at bits 17-22, M >> 4 at bits 24-28.
__device__ __forceinline__ uint32_t idesc_bf16(uint32_t M, uint32_t N) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((N >> 3) << 17) | ((M >> 4) << 24);
}
__device__ __forceinline__ void umma_bf16(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                          uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// 16 bytes global -> shared, of which the first `bytes` (0 .. 16) are read and
// the rest are zeros.
__device__ __forceinline__ void copy16_async(uint32_t dst, const void *src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// An arrival on `bar` once all of this thread's copies so far have landed.
__device__ __forceinline__ void arrive_when_copied(uint64_t *bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
template <int N>
__device__ __forceinline__ void bulk_wait_group_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}

// Byte offset of 16-byte chunk c of row r in a tile of 128-byte rows with the
// 128-byte swizzle.
__device__ __forceinline__ uint32_t sw128(int r, int c) { return r * 128 + ((c ^ (r & 7)) << 4); }

constexpr int kTile = 128;  // tokens of one adapter that a CTA takes

// ---------------------------------------------------------------- shrink

constexpr int kShrinkStages = 6;
constexpr int kShrinkLag = kShrinkStages - 2;  // stages whose copies may be in flight
constexpr int kShrinkThreads = 288;            // 8 copying warps, 1 issuing

struct ShrinkBars {
  uint64_t full[kShrinkStages], empty[kShrinkStages], done;
  uint32_t tmem, abort, never, last;
};

__global__ void __launch_bounds__(kShrinkThreads, 1) lora_shrink_large_kernel(const LoraArgs p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ ShrinkBars bars;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int M = static_cast<int>(p.M), Rp = (p.R + 15) / 16 * 16;
  volatile uint32_t *abort = &bars.abort;
  const uint64_t limit = p.wait_limit_ns;
  const int stage = 128 * 128 + Rp * 128;
  const uint32_t ring = (smem_u32(smem_raw) + 1023u) & ~1023u;
  if (tid == 0) {
    for (int i = 0; i < kShrinkStages; ++i) {
      mbar_init(&bars.full[i], 256);
      mbar_init(&bars.empty[i], 1);
    }
    mbar_init(&bars.done, 1);
    bars.abort = bars.never = 0;
    fence_mbar_init();
  }
  if (warp == 8) {
    tmem_alloc(&bars.tmem, 128);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars.tmem;
  griddep_wait();
  griddep_launch_dependents();
  const Tile t = find_tile<kTile>(p.offsets, p.L, M, blockIdx.x, false);
  const int rank = rank_of(p, t.a);
  const int kb0 = blockIdx.y * p.kb_split;
  const int steps = t.count > 0 && rank > 0 ? min((p.K + 63) / 64, kb0 + p.kb_split) - kb0 : 0;

  if (steps > 0 && warp < 8) {
    // thread: chunk c (8 values) of rows r, r + 32, ... of both operands
    const int r = tid >> 3, c = tid & 7;
    const uint16_t *xr[4], *ar[4];
    uint32_t xb[4], ab[4];  // bytes read of a chunk: 16, or 0 where the row is none
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = r + 32 * i;
      const int tok = row < t.count ? __ldg(p.order + t.start + row) : -1;
      const bool on = tok >= 0 && tok < M;
      xr[i] = on ? p.x + tok * p.ldx : p.x;
      xb[i] = on ? 16 : 0;
      ar[i] = p.a + (static_cast<int64_t>(t.a) * p.R + (row < rank ? row : 0)) * p.K;
      ab[i] = row < rank ? 16 : 0;
    }
    bool ok = true;
    int issued = 0;
    auto give = [&](int s) {  // fault injection: the first stage's wait runs out
      if (!(p.fault && blockIdx.x == 0 && blockIdx.y == 0 && s == 0))
        mbar_arrive(&bars.full[s % kShrinkStages]);
    };
    for (int s = 0; s < steps; ++s) {
      const int st = s % kShrinkStages;
      if (s >= kShrinkStages)
        ok = mbar_wait(&bars.empty[st], (s / kShrinkStages & 1) ^ 1, abort, limit);
      if (!ok) break;
      const uint32_t xs = ring + st * stage, as = xs + 128 * 128;
      const int k = (kb0 + s) * 64 + c * 8;
      const bool in = k < p.K;  // K is a multiple of 16
      const int ko = in ? k : 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) copy16_async(xs + sw128(r + 32 * i, c), xr[i] + ko, in ? xb[i] : 0);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (r + 32 * i < Rp) copy16_async(as + sw128(r + 32 * i, c), ar[i] + ko, in ? ab[i] : 0);
      copies_commit();
      ++issued;
      if (s >= kShrinkLag) {
        copies_wait<kShrinkLag>();
        fence_proxy_async_smem();
        give(s - kShrinkLag);
      }
    }
    copies_wait<0>();
    fence_proxy_async_smem();
    if (ok)
      for (int s = max(0, issued - kShrinkLag); s < issued; ++s) give(s);
  } else if (steps > 0 && lane == 0) {
    const uint32_t idesc = idesc_bf16(128, Rp);
    for (int s = 0; s < steps; ++s) {
      const int st = s % kShrinkStages;
      if (!mbar_wait(&bars.full[st], s / kShrinkStages & 1, abort, limit)) break;
      tc_fence_after();
      const uint64_t xd = sdesc_kmajor_sw128(ring + st * stage);
      const uint64_t ad = sdesc_kmajor_sw128(ring + st * stage + 128 * 128);
#pragma unroll
      for (int k = 0; k < 4; ++k) umma_bf16(tmem, xd + 2 * k, ad + 2 * k, idesc, s > 0 || k > 0);
      umma_commit(&bars.empty[st]);
    }
    umma_commit(&bars.done);
  }
  __syncwarp();
  if (steps > 0 && warp < 4) {
    mbar_wait(&bars.done, 0, abort, limit);
    __syncwarp();
    tc_fence_after();
    const int row = warp * 32 + lane;
    float *out = p.part + (static_cast<int64_t>(blockIdx.y) * p.M + t.start + row) * p.R;
    for (int c0 = 0; c0 < Rp; c0 += 16) {
      uint32_t v[16];
      tmem_ld16(tmem + (static_cast<uint32_t>(warp * 32) << 16) + c0, v);
      tmem_ld_wait();
      if (row < t.count) {
#pragma unroll
        for (int i = 0; i < 16; i += 4)
          if (c0 + i < p.R)
            *reinterpret_cast<uint4 *>(out + c0 + i) = make_uint4(v[i], v[i + 1], v[i + 2], v[i + 3]);
      }
    }
    tc_fence_before();
  }
  if (steps > 0 && warp < 8) {
    // the last of the tile's splits adds them all, in order, and leaves t as the
    // second product's operand: scaled, zeros past the rank, high and low halves
    named_bar_sync(1, 256);
    if (tid == 0) {
      bars.last = gridDim.y == 1 || atom_add_acq_rel_gpu(&p.tickets[blockIdx.x], 1) == gridDim.y - 1;
      if (bars.last && gridDim.y > 1) p.tickets[blockIdx.x] = 0;
    }
    named_bar_sync(1, 256);
    if (bars.last) {
      const float scale = __ldg(p.scales + t.a);
      const int per = Rp / 8;
      for (int i = tid; i < t.count * per; i += 256) {
        const int row = i / per, c = i - row * per;
        float v[8] = {};
        if (c * 8 < p.R) {
          const float *at = p.part + (static_cast<int64_t>(t.start) + row) * p.R + c * 8;
#pragma unroll 4
          for (int s = 0; s < p.splits; ++s) {
            const float4 *q = reinterpret_cast<const float4 *>(at + s * p.M * p.R);
            const float4 f = __ldcg(q), g = __ldcg(q + 1);
            v[0] += f.x, v[1] += f.y, v[2] += f.z, v[3] += f.w;
            v[4] += g.x, v[5] += g.y, v[6] += g.z, v[7] += g.w;
          }
        }
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float x = c * 8 + 2 * j < rank ? v[2 * j] * scale : 0.0f;
          const float y = c * 8 + 2 * j + 1 < rank ? v[2 * j + 1] * scale : 0.0f;
          hi[j] = pack_bf16(x, y);
          lo[j] = pack_bf16(low_half(x, bf16_lo(hi[j])), low_half(y, bf16_hi(hi[j])));
        }
        uint16_t *out = p.t + (static_cast<int64_t>(t.start) + row) * 2 * Rp + c * 8;
        *reinterpret_cast<uint4 *>(out) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4 *>(out + Rp) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      }
    }
  }
  if (steps > 0 && warp == 8 && lane == 0)  // the MMAs are done before the memory is given up
    mbar_wait(&bars.done, 0, &bars.never, limit);
  __syncthreads();
  if (tid == 0 && *abort) atomicMax(p.status, kStatusTimeout);
  if (warp == 8) tmem_dealloc(tmem, 128);
}

// ---------------------------------------------------------------- expand

constexpr int kExpandThreads = 416;  // 8 row warps, 1 issuing, 4 copying B
constexpr int kRowThreads = 256;
constexpr int kBlockCols = 128;
constexpr int kWarpBytes = 32 * kBlockCols * 2;  // a warp's rows of a block: two halves of 64 columns
constexpr int kHalfBytes = kWarpBytes / 2;
constexpr int kBufBytes = 4 * kWarpBytes;
constexpr int kMaxBStages = 3;

struct ExpandBars {
  uint64_t base[2][2][4];  // by row group, its buffer, warp
  uint64_t bfull[kMaxBStages], bempty[kMaxBStages];
  uint64_t dfull[2], dempty[2];
  uint64_t sfull, done;
  uint32_t tmem, abort, never;
};

// Tiles of all segments (and of the rows without an adapter), by one warp.
__device__ int count_tiles(const int *offsets, int L, int M, bool rest) {
  const int lane = threadIdx.x & 31;
  auto bound = [&](int k) { return k > L ? M : min(max(__ldg(offsets + k), 0), M); };
  int n = 0;
  for (int k = lane; k < L + (rest ? 1 : 0); k += 32)
    n += (max(bound(k + 1) - bound(k), 0) + kTile - 1) / kTile;
  return __reduce_add_sync(0xFFFFFFFFu, n);
}

// KT: 64-wide tiles of the rank (R <= 64 KT); NB: base buffers of a row group
template <int KT, int NB>
__global__ void __launch_bounds__(kExpandThreads, 1)
    lora_expand_large_kernel(const __grid_constant__ CUtensorMap base8,
                             const __grid_constant__ CUtensorMap y8,
                             const __grid_constant__ CUtensorMap base32,
                             const __grid_constant__ CUtensorMap y32, const LoraArgs p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ ExpandBars bars;
  constexpr int kOperand = KT * 128 * 128;  // bytes of one 128-row operand
  constexpr int kBStages = KT == 1 ? 3 : 2;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int M = static_cast<int>(p.M), Rp = (p.R + 15) / 16 * 16;
  volatile uint32_t *abort = &bars.abort;
  const uint64_t limit = p.wait_limit_ns;
  uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t *s_hi = smem, *s_lo = smem + kOperand, *b_ring = smem + 2 * kOperand;
  uint8_t *base_ring = b_ring + kBStages * kOperand;
  if (tid == 0) {
    for (int i = 0; i < 16; ++i) mbar_init(&bars.base[i >> 3][i >> 2 & 1][i & 3], 32);
    for (int i = 0; i < kBStages; ++i) {
      mbar_init(&bars.bfull[i], 128);
      mbar_init(&bars.bempty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.dfull[i], 1);
      mbar_init(&bars.dempty[i], 4);
    }
    mbar_init(&bars.sfull, kRowThreads);
    mbar_init(&bars.done, 1);
    bars.abort = bars.never = 0;
    fence_mbar_init();
  }
  if (warp == 8) {
    tmem_alloc(&bars.tmem, 256);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars.tmem;
  griddep_launch_dependents();
  // (as in the direct form, all but t is visible here already)
  const int tiles = count_tiles(p.offsets, p.L, M, p.copy_rest != 0);
  const int nblk = (p.N + kBlockCols - 1) / kBlockCols;
  const int64_t work = static_cast<int64_t>(tiles) * nblk;
  const int64_t w0 = work * blockIdx.x / gridDim.x, w1 = work * (blockIdx.x + 1) / gridDim.x;

  if (warp < 8) {
    // ---- rows: two groups of four warps take the blocks in turn, each with its
    // own product buffer and base buffers; a thread has a token of the tile
    const int grp = warp >> 2, wg = warp & 3, row = tid & 127;
    const uint32_t lanes = static_cast<uint32_t>(wg * 32) << 16;
    uint8_t *const mine = base_ring + grp * NB * kBufBytes + wg * kWarpBytes;
    const int gr = lane & 7, g8 = lane & 24;  // row of its eight, and those
    const uint32_t peers = 0xFFu << g8;
    int dph = 0;            // the product buffer's phase
    int bufs = 0, seen = 0; // blocks whose base was asked for, and those that arrived
    int64_t q = 0;          // blocks of this CTA so far, both groups'
    bool ok = true;         // a thread that gave up waiting goes on to the barriers alone
    griddep_wait();
    for (int64_t w = w0; w < w1;) {
      const int tile = static_cast<int>(w / nblk), blk0 = static_cast<int>(w - static_cast<int64_t>(tile) * nblk);
      const int blk1 = static_cast<int>(w1 - w < nblk - blk0 ? blk0 + (w1 - w) : nblk);
      w += blk1 - blk0;
      const Tile t = find_tile<kTile>(p.offsets, p.L, M, tile, p.copy_rest != 0);
      const int rank = rank_of(p, t.a);
      int tok = row < t.count ? __ldg(p.order + t.start + row) : -1;
      if (tok >= M) tok = -1;
      // 32 tokens that lie next to each other move as two boxes of 64 columns,
      // 128-byte swizzled, a thread's two instructions; so do eight; others go by
      // plain 16-byte accesses of their eight lanes, held in the same way (a bulk
      // copy a row costs the copy unit about 10 ns: 256 of them a block took 2.4
      // us against the 1.5 us that HBM needs)
      const int tok0 = __shfl_sync(0xFFFFFFFFu, tok, 0), tok8 = __shfl_sync(0xFFFFFFFFu, tok, g8);
      const bool all = __ballot_sync(0xFFFFFFFFu, tok >= 0 && tok == tok0 + lane) == 0xFFFFFFFFu;
      const uint32_t next = __ballot_sync(0xFFFFFFFFu, tok >= 0 && tok == tok8 + gr);
      const bool box = (next >> g8 & 0xFFu) == 0xFFu;
      const bool lead = all ? lane == 0 : box && gr == 0;  // issues for its rows
      auto ask = [&](int blk) {  // base of block blk into the next buffer
        const int b = bufs % NB;
        uint64_t *bar = &bars.base[grp][b][wg];
        uint8_t *to = mine + b * kBufBytes;
        if (box) {
          if (lead) {
            const CUtensorMap *map = all ? &base32 : &base8;
            mbar_arrive_expect_tx(bar, all ? kWarpBytes : kWarpBytes / 4);
            tma_load_2d(to + g8 * 128, map, bar, blk * kBlockCols, tok);
            tma_load_2d(to + kHalfBytes + g8 * 128, map, bar, blk * kBlockCols + 64, tok);
          } else {
            mbar_arrive(bar);
          }
        } else {
          const int cols = min(kBlockCols, p.N - blk * kBlockCols);
#pragma unroll
          for (int r = 0; r < 8; ++r) {
            const int rt = __shfl_sync(peers, tok, g8 + r);
            if (rt < 0) continue;
            const uint16_t *from = p.base + rt * p.ldbase + blk * kBlockCols;
#pragma unroll
            for (int c = gr; c < kBlockCols / 8; c += 8)
              if (c * 8 < cols)
                copy16_async(smem_u32(to) + (c >> 3) * kHalfBytes + sw128(g8 + r, gr), from + c * 8, 16);
          }
          arrive_when_copied(bar);
        }
        ++bufs;
      };
      const int first = blk0 + (static_cast<int>(q ^ grp) & 1);
      int asked = first;
      bulk_wait_group_read<0>();  // the buffers' last stores have read them
      __syncwarp();
      for (; ok && asked < blk1 && asked < first + 2 * NB; asked += 2) ask(asked);
      // t's rows of the tile, once the last tile's products are done
      named_bar_sync(1, kRowThreads);
      if (rank > 0) {
        const int per = (rank + 15) / 16 * 2;
        for (int i = tid; i < 128 * per; i += kRowThreads) {
          const int r = i / per, c = i - r * per;
          const uint32_t off = (c >> 3) * 128 * 128 + sw128(r, c & 7);
          const uint16_t *from = p.t + (static_cast<int64_t>(t.start) + (r < t.count ? r : 0)) * 2 * Rp + c * 8;
          const uint32_t bytes = r < t.count ? 16 : 0;
          copy16_async(smem_u32(s_hi) + off, from, bytes);
          copy16_async(smem_u32(s_lo) + off, from + Rp, bytes);
        }
        copies_commit();
        copies_wait<0>();
        fence_proxy_async_smem();
        mbar_arrive(&bars.sfull);
      }
      for (int blk = first; blk < blk1; blk += 2) {
        const int b = seen % NB;
        if (ok) ok = mbar_wait(&bars.base[grp][b][wg], seen / NB & 1, abort, limit);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) continue;
        ++seen;
        uint8_t *const my = mine + b * kBufBytes;
        const int cols = min(kBlockCols, p.N - blk * kBlockCols);
        if (rank > 0) {
          mbar_wait(&bars.dfull[grp], dph, abort, limit);
          __syncwarp();
          dph ^= 1;
          tc_fence_after();
          uint32_t v[2][32];
          tmem_ld32(tmem + lanes + grp * 128, v[0]);
#pragma unroll
          for (int c0 = 0; c0 < kBlockCols; c0 += 32) {
            tmem_ld_wait();
            if (c0 + 32 < kBlockCols) {
              tmem_ld32(tmem + lanes + grp * 128 + c0 + 32, v[(c0 / 32 + 1) & 1]);
            } else {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&bars.dempty[grp]);
            }
            const uint32_t *d = v[c0 / 32 & 1];
            // chunk c0 / 8 + i of this row
            uint4 *at[4], h[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int c = c0 / 8 + i;
              at[i] = reinterpret_cast<uint4 *>(
                  my + (c >> 3) * kHalfBytes + sw128(lane, c & 7));
              h[i] = *at[i];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t hw[4] = {h[i].x, h[i].y, h[i].z, h[i].w};
              uint32_t o[4];
#pragma unroll
              for (int j = 0; j < 4; ++j)
                o[j] = pack_bf16(bf16_lo(hw[j]) + __uint_as_float(d[i * 8 + 2 * j]),
                                 bf16_hi(hw[j]) + __uint_as_float(d[i * 8 + 2 * j + 1]));
              *at[i] = make_uint4(o[0], o[1], o[2], o[3]);
            }
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (box) {
          if (lead) {
            const CUtensorMap *map = all ? &y32 : &y8;
            tma_store_2d(map, my + g8 * 128, blk * kBlockCols, tok);
            if (cols > 64) tma_store_2d(map, my + kHalfBytes + g8 * 128, blk * kBlockCols + 64, tok);
          }
        } else {
#pragma unroll
          for (int r = 0; r < 8; ++r) {
            const int rt = __shfl_sync(peers, tok, g8 + r);
            if (rt < 0) continue;
            uint16_t *out = p.y + rt * p.ldy + blk * kBlockCols;
#pragma unroll
            for (int c = gr; c < kBlockCols / 8; c += 8)
              if (c * 8 < cols)
                *reinterpret_cast<uint4 *>(out + c * 8) =
                    *reinterpret_cast<const uint4 *>(my + (c >> 3) * kHalfBytes + sw128(g8 + r, gr));
          }
        }
        bulk_commit_group();
        if (asked < blk1) {  // into the same buffer, which the store leaves within 0.1 us
          bulk_wait_group_read<0>();
          __syncwarp();
          ask(asked);
          asked += 2;
        }
      }
      q += blk1 - blk0;
    }
    // copies still in flight land before the memory is given up
    copies_wait<0>();
    for (; seen < bufs; ++seen)
      mbar_wait(&bars.base[grp][seen % NB][wg], seen / NB & 1, &bars.never, limit);
    bulk_wait_group0();
  } else if (warp == 8) {
    // ---- MMAs: t's high and low halves against the same rows of B
    const uint32_t idesc = idesc_bf16(128, kBlockCols);
    const uint64_t hd = sdesc_kmajor_sw128(smem_u32(s_hi)), ld = sdesc_kmajor_sw128(smem_u32(s_lo));
    int st = 0, ph = 0, sph = 0;
    uint32_t dph = 0;  // the product buffers' phases, a bit each
    int64_t q = 0;     // blocks so far: block q goes to buffer q % 2
    bool ok = true;
    for (int64_t w = w0; w < w1 && ok;) {
      const int tile = static_cast<int>(w / nblk), blk0 = static_cast<int>(w - static_cast<int64_t>(tile) * nblk);
      const int blk1 = static_cast<int>(w1 - w < nblk - blk0 ? blk0 + (w1 - w) : nblk);
      w += blk1 - blk0;
      const Tile t = find_tile<kTile>(p.offsets, p.L, M, tile, p.copy_rest != 0);
      const int rank = rank_of(p, t.a), ks = (rank + 15) / 16;
      q += blk1 - blk0;
      if (rank == 0) continue;
      if (lane == 0) {
        ok = mbar_wait(&bars.sfull, sph, abort, limit);
        for (int blk = blk0; blk < blk1 && ok; ++blk) {
          const int db = static_cast<int>(q - (blk1 - blk)) & 1;
          ok = mbar_wait(&bars.bfull[st], ph, abort, limit) &&
               mbar_wait(&bars.dempty[db], (dph >> db & 1) ^ 1, abort, limit);
          if (!ok) break;
          dph ^= 1u << db;
          tc_fence_after();
          const uint64_t bd = sdesc_kmajor_sw128(smem_u32(b_ring + st * kOperand));
          for (int k = 0; k < ks; ++k) {
            const uint64_t off = (k >> 2) * (128 * 128 / 16) + (k & 3) * 2;
            umma_bf16(tmem + db * 128, hd + off, bd + off, idesc, k > 0);
            umma_bf16(tmem + db * 128, ld + off, bd + off, idesc, 1);
          }
          umma_commit(&bars.bempty[st]);
          umma_commit(&bars.dfull[db]);
          if (++st == kBStages) st = 0, ph ^= 1;
        }
      }
      sph ^= 1;
      ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
    }
    if (lane == 0) {
      umma_commit(&bars.done);
      mbar_wait(&bars.done, 0, &bars.never, limit);
    }
    __syncwarp();
  } else {
    // ---- B_a's rows: thread = chunk (8 ranks) c of rows r, r + 16, ...
    const int bt = tid - 288, r = bt >> 3, c = bt & 7;
    int st = 0, ph = 1, filled = 0, given = 0;
    bool ok = true;
    for (int64_t w = w0; w < w1 && ok;) {
      const int tile = static_cast<int>(w / nblk), blk0 = static_cast<int>(w - static_cast<int64_t>(tile) * nblk);
      const int blk1 = static_cast<int>(w1 - w < nblk - blk0 ? blk0 + (w1 - w) : nblk);
      w += blk1 - blk0;
      const Tile t = find_tile<kTile>(p.offsets, p.L, M, tile, p.copy_rest != 0);
      const int rank = rank_of(p, t.a);
      if (rank == 0) continue;
      const uint16_t *b = p.b + static_cast<int64_t>(t.a) * p.N * p.R;
      for (int blk = blk0; blk < blk1; ++blk) {
        ok = mbar_wait(&bars.bempty[st], ph, abort, limit);
        if (!ok) break;
        const uint32_t to = smem_u32(b_ring + st * kOperand);
#pragma unroll
        for (int kt = 0; kt < KT; ++kt) {
          const int k = kt * 64 + c * 8;
          if (k >= (rank + 15) / 16 * 16) continue;  // a step that no MMA takes
          const int bytes = min(max(rank - k, 0), 8) * 2;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int n = blk * kBlockCols + r + 16 * i;
            const bool in = n < p.N && bytes > 0;
            copy16_async(to + kt * 128 * 128 + sw128(r + 16 * i, c),
                         in ? b + static_cast<int64_t>(n) * p.R + k : b, in ? bytes : 0);
          }
        }
        copies_commit();
        ++filled;
        if (++st == kBStages) st = 0, ph ^= 1;
        if (filled - given == 2) {  // the one before has landed
          copies_wait<1>();
          fence_proxy_async_smem();
          mbar_arrive(&bars.bfull[given++ % kBStages]);
        }
      }
    }
    copies_wait<0>();
    fence_proxy_async_smem();
    for (; given < filled; ++given) mbar_arrive(&bars.bfull[given % kBStages]);
  }
  __syncthreads();
  if (tid == 0 && *abort) atomicMax(p.status, kStatusTimeout);
  if (warp == 8) tmem_dealloc(tmem, 256);
}

}  // namespace

cudaError_t launch_lora_large(const LoraArgs &a, int num_sms, cudaStream_t st) {
  const int64_t full = (a.M + kTile - 1) / kTile;
  const int64_t tiles = full + a.L < a.M ? full + a.L : a.M;
  const int Rp = (a.R + 15) / 16 * 16;
  const int smem1 = kShrinkStages * (128 * 128 + Rp * 128) + 1024;
  cudaError_t e = allow_smem<lora_shrink_large_kernel>(kShrinkStages * (128 * 128 * 2) + 1024);
  if (e != cudaSuccess) return e;
  e = launch_pdl(lora_shrink_large_kernel, dim3(static_cast<unsigned>(tiles), a.splits),
                 dim3(kShrinkThreads), smem1, st, a);
  if (e != cudaSuccess) return e;
  CUtensorMap base8, y8, base32, y32;
  if (!make_bf16_map(&base8, a.base, a.M, a.N, a.ldbase, 64, 8) ||
      !make_bf16_map(&y8, a.y, a.M, a.N, a.ldy, 64, 8) ||
      !make_bf16_map(&base32, a.base, a.M, a.N, a.ldbase, 64, 32) ||
      !make_bf16_map(&y32, a.y, a.M, a.N, a.ldy, 64, 32))
    return cudaErrorInvalidValue;
  auto expand = [&](auto kt) {
    constexpr int KT = decltype(kt)::value, NB = KT == 1 ? 2 : 1;
    constexpr int smem = (2 + (KT == 1 ? 3 : 2)) * KT * 128 * 128 + 2 * NB * kBufBytes + 1024;
    cudaError_t r = allow_smem<lora_expand_large_kernel<KT, NB>>(smem);
    if (r != cudaSuccess) return r;
    return launch_pdl(lora_expand_large_kernel<KT, NB>, dim3(num_sms), dim3(kExpandThreads), smem,
                      st, base8, y8, base32, y32, a);
  };
  return a.R <= 64 ? expand(std::integral_constant<int, 1>{})
                   : expand(std::integral_constant<int, 2>{});
}

}  // namespace fp8bq
