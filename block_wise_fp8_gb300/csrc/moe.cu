// moe.cu -- a whole mixture-of-experts layer for at most 64 tokens in one
// kernel, over block-FP8 experts w13 [E, 2I, H] (gate rows, then up rows) and
// w2 [E, H, I] with one FP32 128 x 128 scale grid each, the weights of the
// grouped GEMM.
//
//   route   per token the top-k logits (or ids and weights from the caller)
//   x       group-128 quantisation, s = max|x| * RN(1 / 448), q = RNE(x / s)
//   g, u    = sum_b P_b s_x[b] s_13[b],  P_b the FP32 tensor-core sum of K block b
//   h       = g / (1 + exp(-g)) * u (FP32), group-128 quantised in the same way
//   o       = sum_b P_b s_h[b] s_2[b]
//   y       = BF16(sum_k w_k o_k)
//
// Bound by HBM: the weights of every expert that a token chose are read once
// (3 I H bytes each); with so few tokens nothing else counts but the latency of
// the steps that depend on one another.  So the layer is one persistent
// kernel, one CTA an SM (a cooperative launch, since CTAs wait on one another),
// and its weight copies never wait for activations: a warp streams the weight
// tiles of both products, in order, through a ring in shared memory, while a
// second warp adds the activation tiles to the same stages once the CTAs that
// produce them have published them.  Across each dependency (quantised x, the
// experts' h) the ring fills with weights instead of draining.
//
// Both products are cut into steps of two 128 x 128 weight tiles that share an
// activation tile (gate and up rows of 128 hidden columns; two tiles of 128
// output rows), and every CTA takes an equal, contiguous run of steps: cuts
// fall inside a sum over K.  The sums cut in the first product meet in the
// workspace, where the last CTA to finish adds them in CTA order; in the second
// product the partial sums of all experts of an output tile add up in shared
// memory, weighted, and meet once a tile.  All orders are fixed by the sizes
// and the routing, so results repeat bit for bit.
//
// The tensor core sees the weights as the 128 rows of A and up to NT tokens as
// the columns of B (tcgen05.mma, M = 128, N = 16 or 32).  Tokens of one expert
// beyond NT form a further entry that reads the weights again, from L2.
//
// Routing is computed by every CTA for itself: at these sizes that is cheaper
// than one CTA's result handed to the others.
#include "common.cuh"
#include "ptx.cuh"
#include "quant_math.cuh"

namespace fp8bq {
namespace {

constexpr int kMoeThreads = 384;  // 4 warps of roles, 8 of the epilogue
constexpr int kEpi = 256;
constexpr int kSlots = 8;         // TMEM partial-sum buffers of two 32-column tiles
constexpr int kTileBytes = 128 * 128;
constexpr int kMaxRing = 8;
// The codes never leave the layer, so the scale is a product with the binary32
// reciprocal, not the quantisers' division: it may differ from theirs by one
// binary32 step, which is nothing to a code's 2^-4.
constexpr float kInv448 = 1.0f / 448.0f;

__device__ __forceinline__ void fence_proxy_async_all() {
  asm volatile("fence.proxy.async;" ::: "memory");
}
__device__ __forceinline__ uint32_t ld_acquire_gpu(const uint32_t *p) {
  uint32_t v;
  asm volatile("ld.acquire.gpu.global.b32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ void red_release_gpu(uint32_t *p, uint32_t v) {
  asm volatile("red.release.gpu.global.add.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}

// Bounded wait until *p reaches `target` (counters only grow during a launch).
__device__ __forceinline__ bool wait_count(const uint32_t *p, uint32_t target,
                                           volatile uint32_t *abort, uint64_t limit_ns) {
  if (ld_acquire_gpu(p) >= target) return true;
  const uint64_t t0 = global_timer_ns();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 32; ++i)
      if (ld_acquire_gpu(p) >= target) return true;
    if (*abort) return false;
    if (global_timer_ns() - t0 > limit_ns) {
      *abort = 1u;
      return false;
    }
  }
}

__device__ __forceinline__ uint16_t bf16_bits(float v) {
  uint16_t r;
  asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(r) : "f"(v));
  return r;
}

struct MoeBars {
  uint64_t full_w[kMaxRing], full_b[kMaxRing], empty[kMaxRing];
  uint64_t tfull[kSlots], tempty[kSlots];
  uint64_t drain;
  uint32_t tmem;
  uint32_t abort, never;  // never stays 0
  uint32_t flag;
  int entries;
};

// Expert entry: expert, first row of its tokens in the pair-ordered buffers,
// tokens (at most NT)
struct Entry {
  int e, row, n;
};

// The run of steps of CTA c out of `steps` steps dealt to `parts` CTAs
// (parts <= steps, so that none is empty), and the CTA that has a step.
__device__ __forceinline__ int run_begin(int c, int steps, int parts) {
  return static_cast<int>(static_cast<int64_t>(c) * steps / parts);
}
__device__ __forceinline__ int owner_of(int step, int steps, int parts) {
  return static_cast<int>((static_cast<int64_t>(step + 1) * parts - 1) / steps);
}

// ---------------------------------------------------------------- routing

// A token's choice by one warp: ids into id[0..topk), weights into w[0..topk).
// Lanes hold the keys of experts lane, lane + 32, ...; a chosen key becomes
// -inf.  NaN and -inf logits are never chosen (id -1, weight 0); +inf counts
// as the largest finite number.
__device__ void route_token(const MoeArgs &a, int t, short *id, float *w) {
  constexpr int R = kMaxMoeExperts / 32;
  const int lane = threadIdx.x & 31;
  const float kNone = -INFINITY;
  const float *row = a.logits + static_cast<int64_t>(t) * a.E;
  const bool by_bias = a.bias != nullptr;
  float key[R];
  float top = kNone;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    key[r] = kNone;
    if (r * 32 < a.E) {
      const int e = r * 32 + lane;
      const float l = e < a.E ? __ldg(row + e) : kNone;
      key[r] = l == l ? fminf(l, 3.402823466e38f) : kNone;
      top = fmaxf(top, key[r]);
    }
  }
  float denom = 1.0f;
  if (a.score == 0) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
    float s = 0.0f;
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (r * 32 < a.E && key[r] > kNone) s += expf(key[r] - top);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
    denom = s;
  }
  // chosen by sigmoid + bias; without a bias the order is the logits' own
  if (by_bias) {
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (r * 32 < a.E && key[r] > kNone)
        key[r] = 1.0f / (1.0f + expf(-key[r])) + __ldg(a.bias + r * 32 + lane);
  }
  float sum = 0.0f;
  for (int k = 0; k < a.topk; ++k) {
    float best = kNone;
    int at = 1 << 20;
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (r * 32 < a.E && key[r] > best) best = key[r], at = r * 32 + lane;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      const float ob = __shfl_xor_sync(0xFFFFFFFFu, best, d);
      const int oa = __shfl_xor_sync(0xFFFFFFFFu, at, d);
      if (ob > best || (ob == best && oa < at)) best = ob, at = oa;
    }
    if (by_bias && best > kNone) {
      // Keys this close may be ordered by binary32 rounding (a few 2^-24 of a
      // sigmoid below 1 and of the sum): such a choice is made in 64 bits.
      const float near = best - (1e-6f + 4e-7f * fabsf(best));
      int close = 0;
#pragma unroll
      for (int r = 0; r < R; ++r) close += r * 32 < a.E && key[r] >= near ? 1 : 0;
      if (__reduce_add_sync(0xFFFFFFFFu, close) > 1) {
        double bd = -1e300;
        int bat = 1 << 20;
#pragma unroll 1
        for (int r = 0; r * 32 < a.E; ++r) {
          const int e = r * 32 + lane;
          float kr = kNone;
#pragma unroll
          for (int i = 0; i < R; ++i)
            if (i == r) kr = key[i];
          if (kr >= near) {
            const double l = fminf(__ldg(row + e), 3.402823466e38f);
            const double v = 1.0 / (1.0 + exp(-l)) + static_cast<double>(__ldg(a.bias + e));
            if (v > bd) bd = v, bat = e;
          }
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) {
          const double ob = __shfl_xor_sync(0xFFFFFFFFu, bd, d);
          const int oa = __shfl_xor_sync(0xFFFFFFFFu, bat, d);
          if (ob > bd || (ob == bd && oa < bat)) bd = ob, bat = oa;
        }
        at = bat;
      }
    }
    const bool none = best == kNone;
    float v = 0.0f;
    if (!none) {
      const float l = fminf(__ldg(row + at), 3.402823466e38f);
      v = a.score == 0 ? expf(l - top) / denom : 1.0f / (1.0f + expf(-l));
#pragma unroll
      for (int r = 0; r < R; ++r)
        if (r == at >> 5 && lane == (at & 31)) key[r] = kNone;
    }
    sum += v;
    if (lane == 0) {
      id[k] = none ? -1 : static_cast<short>(at);
      w[k] = v;
    }
  }
  __syncwarp();
  if (lane < a.topk) {
    float v = w[lane];
    if (a.renorm) v = sum > 0.0f ? v / sum : 0.0f;
    w[lane] = v * a.scale;
  }
}

// ---------------------------------------------------------------- the kernel

template <int NT>
__global__ void __launch_bounds__(kMoeThreads, 1)
    moe_layer_kernel(const __grid_constant__ CUtensorMap map13,
                     const __grid_constant__ CUtensorMap map2,
                     const __grid_constant__ CUtensorMap mapx,
                     const __grid_constant__ CUtensorMap maph, const MoeArgs a) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ MoeBars bars;
  constexpr int kStage = 2 * kTileBytes + NT * 128;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int cta = blockIdx.x, ctas = gridDim.x;
  const uint64_t limit = a.wait_limit_ns;
  volatile uint32_t *abort = &bars.abort;
  volatile uint32_t *never = &bars.never;
  const int pairs = a.M * a.topk;

  uint8_t *ring = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  float *ysum = reinterpret_cast<float *>(ring + a.stages * kStage);  // [M][256], or [NT][128]
  const int ysum_floats = max(a.M * 256, NT * 128);
  float *wgt = ysum + ysum_floats;                          // [pairs]
  Entry *ent = reinterpret_cast<Entry *>(wgt + pairs);      // [max_entries]
  int *eoff = reinterpret_cast<int *>(ent + a.max_entries);  // [E]: count, then first row
  short *ids = reinterpret_cast<short *>(eoff + a.E);       // [pairs]
  short *row_of = ids + pairs;                              // [pairs]: place in expert, then row
  short *pair_of = row_of + pairs;                          // [pairs], by row

  if (tid == 0) {
    for (int i = 0; i < a.stages; ++i) {
      mbar_init(&bars.full_w[i], 1);
      mbar_init(&bars.full_b[i], 1);
      mbar_init(&bars.empty[i], 1);
    }
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&bars.tfull[i], 1);
      mbar_init(&bars.tempty[i], kEpi / 32);
    }
    mbar_init(&bars.drain, 1);
    bars.abort = 0;
    bars.never = 0;
    fence_mbar_init();
    tma_prefetch_desc(&map13);
    tma_prefetch_desc(&map2);
    tma_prefetch_desc(&mapx);
    tma_prefetch_desc(&maph);
  }
  if (warp == 1) {
    tmem_alloc(&bars.tmem, 512);
    tmem_relinquish();
  }
  for (int e = tid; e < a.E; e += kMoeThreads) eoff[e] = 0;

  // ---- routing, by every CTA
  if (a.logits) {
    for (int t = warp; t < a.M; t += kMoeThreads / 32)
      route_token(a, t, ids + t * a.topk, wgt + t * a.topk);
  } else {
    for (int p = tid; p < pairs; p += kMoeThreads) {
      const int e = __ldg(a.ids_in + p);
      ids[p] = e >= 0 && e < a.E ? static_cast<short>(e) : -1;
      wgt[p] = __ldg(a.w_in + p);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) {
    // place of each pair among its expert's, in pair order
    for (int p0 = 0; p0 < pairs; p0 += 32) {
      const int p = p0 + lane;
      const int e = p < pairs ? ids[p] : -1;
      const uint32_t same = __match_any_sync(0xFFFFFFFFu, e);
      const uint32_t lower = same & ((1u << lane) - 1u);
      int before = 0;
      if (e >= 0) before = eoff[e];
      __syncwarp();
      if (e >= 0) {
        row_of[p] = static_cast<short>(before + __popc(lower));
        if (lower == 0) eoff[e] = before + __popc(same);
      }
      __syncwarp();
    }
    // entries and first rows, expert by expert
    int rows = 0, n_ent = 0;
    for (int e0 = 0; e0 < a.E; e0 += 32) {
      const int e = e0 + lane;
      const int n = e < a.E ? eoff[e] : 0;
      const int e_own = (n + NT - 1) / NT;
      int rr = n, ee = e_own;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int v = __shfl_up_sync(0xFFFFFFFFu, rr, d);
        const int u = __shfl_up_sync(0xFFFFFFFFu, ee, d);
        if (lane >= d) rr += v, ee += u;
      }
      const int first = rows + rr - n;
      if (e < a.E) eoff[e] = first;
      for (int i = 0; i < e_own; ++i)
        ent[n_ent + ee - e_own + i] = Entry{e, first + i * NT, min(NT, n - i * NT)};
      rows += __shfl_sync(0xFFFFFFFFu, rr, 31);
      n_ent += __shfl_sync(0xFFFFFFFFu, ee, 31);
    }
    if (lane == 0) bars.entries = n_ent;
  }
  __syncthreads();
  for (int p = tid; p < pairs; p += kMoeThreads) {
    const int e = ids[p];
    if (e >= 0) {
      const int r = eoff[e] + row_of[p];
      row_of[p] = static_cast<short>(r);
      pair_of[r] = static_cast<short>(p);
    }
    if (cta == 0) {
      if (a.ids_out) a.ids_out[p] = e;
      if (a.w_out) a.w_out[p] = wgt[p];
    }
  }
  __syncthreads();

  const int A = bars.entries;
  const int KB1 = (a.H + 127) / 128, G1 = a.I / 128, KB2 = G1, J = (a.H + 255) / 256;
  const int S1 = A * G1 * KB1, S2 = J * A * KB2;
  const int P1 = min(ctas, S1), P2 = min(ctas, S2);
  const int b1 = cta < P1 ? run_begin(cta, S1, P1) : 0, e1 = cta < P1 ? run_begin(cta + 1, S1, P1) : 0;
  const int b2 = cta < P2 ? run_begin(cta, S2, P2) : 0, e2 = cta < P2 ? run_begin(cta + 1, S2, P2) : 0;
  const uint32_t tmem = bars.tmem;
  uint32_t *const all_quant = a.sync;           // CTAs whose share of x is quantised
  uint32_t *const done = a.sync + 1;            // CTAs about to leave
  uint32_t *const tile_cnt = a.sync + 32;       // [J]
  uint32_t *const ready = tile_cnt + J;         // [entries]: hidden groups published
  uint32_t *const unit_cnt = ready + a.max_entries;  // [entries * G1]

  if (warp == 0) {
    if (lane == 0) {  // ---- weight tiles
      int it = 0;
      bool ok = true;
      for (int s = b1; s < e1 && ok; ++s, ++it) {
        const int u = s / KB1, kb = s - u * KB1, ei = u / G1, g = u - ei * G1;
        const int st = it % a.stages;
        ok = mbar_wait(&bars.empty[st], ((it / a.stages) & 1) ^ 1, abort, limit);
        if (!ok) break;
        if (a.fault && cta == 0 && it == 0) continue;  // fault injection: this wait runs out
        uint8_t *dst = ring + st * kStage;
        const int r = ent[ei].e * 2 * a.I + g * 128;
        mbar_arrive_expect_tx(&bars.full_w[st], 2 * kTileBytes);
        tma_load_2d(dst, &map13, &bars.full_w[st], kb * 128, r);
        tma_load_2d(dst + kTileBytes, &map13, &bars.full_w[st], kb * 128, r + a.I);
      }
      for (int s = b2; s < e2 && ok; ++s, ++it) {
        const int u = s / KB2, kb = s - u * KB2, j = u / A, ei = u - j * A;
        const int st = it % a.stages;
        ok = mbar_wait(&bars.empty[st], ((it / a.stages) & 1) ^ 1, abort, limit);
        if (!ok) break;
        uint8_t *dst = ring + st * kStage;
        const int r = ent[ei].e * a.H + j * 256;
        const bool two = j * 256 + 128 < a.H;
        mbar_arrive_expect_tx(&bars.full_w[st], two ? 2 * kTileBytes : kTileBytes);
        tma_load_2d(dst, &map2, &bars.full_w[st], kb * 128, r);
        if (two) tma_load_2d(dst + kTileBytes, &map2, &bars.full_w[st], kb * 128, r + 128);
      }
      if (!ok)  // let the copies in flight land before this CTA's memory is given up
        for (int i = max(a.fault && cta == 0 ? 1 : 0, it - a.stages); i < it; ++i)
          mbar_wait(&bars.full_w[i % a.stages], (i / a.stages) & 1, never, limit);
    }
    __syncwarp();
  } else if (warp == 2) {
    if (lane == 0) {  // ---- activation tiles
      int it = 0;
      bool ok = true;
      if (b1 < e1) ok = wait_count(all_quant, ctas, abort, limit);
      fence_proxy_async_all();
      for (int s = b1; s < e1 && ok; ++s, ++it) {
        const int u = s / KB1, kb = s - u * KB1, ei = u / G1;
        const int st = it % a.stages;
        ok = mbar_wait(&bars.empty[st], ((it / a.stages) & 1) ^ 1, abort, limit);
        if (!ok) break;
        uint8_t *dst = ring + st * kStage + 2 * kTileBytes;
        const Entry en = ent[ei];
        const int boxes = (en.n + 15) / 16;
        mbar_arrive_expect_tx(&bars.full_b[st], boxes * 2048);
        for (int i = 0; i < boxes; ++i)
          tma_load_2d(dst + i * 2048, &mapx, &bars.full_b[st], kb * 128, en.row + i * 16);
      }
      for (int s = b2; s < e2 && ok; ++s, ++it) {
        const int u = s / KB2, kb = s - u * KB2, ei = u % A;
        const int st = it % a.stages;
        if (s == b2 || kb == 0) {
          ok = wait_count(&ready[ei], G1, abort, limit);
          fence_proxy_async_all();
          if (!ok) break;
        }
        ok = mbar_wait(&bars.empty[st], ((it / a.stages) & 1) ^ 1, abort, limit);
        if (!ok) break;
        uint8_t *dst = ring + st * kStage + 2 * kTileBytes;
        const Entry en = ent[ei];
        const int boxes = (en.n + 15) / 16;
        mbar_arrive_expect_tx(&bars.full_b[st], boxes * 2048);
        for (int i = 0; i < boxes; ++i)
          tma_load_2d(dst + i * 2048, &maph, &bars.full_b[st], kb * 128, en.row + i * 16);
      }
      if (!ok)
        for (int i = max(0, it - a.stages); i < it; ++i)
          mbar_wait(&bars.full_b[i % a.stages], (i / a.stages) & 1, never, limit);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {  // ---- MMAs
      int it = 0;
      bool ok = true;
      auto step = [&](int n, bool two) {
        const int st = it % a.stages, sl = it % kSlots;
        if (!mbar_wait(&bars.tempty[sl], ((it / kSlots) & 1) ^ 1, abort, limit) ||
            !mbar_wait(&bars.full_w[st], (it / a.stages) & 1, abort, limit) ||
            !mbar_wait(&bars.full_b[st], (it / a.stages) & 1, abort, limit))
          return false;
        tc_fence_after();
        const uint32_t base = smem_u32(ring + st * kStage);
        const uint32_t idesc = idesc_f8f6f4_e4m3(128, (n + 15) / 16 * 16);
        const uint64_t bd = sdesc_kmajor_sw128(base + 2 * kTileBytes);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (t == 1 && !two) break;
          const uint64_t ad = sdesc_kmajor_sw128(base + t * kTileBytes);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            umma_f8f6f4(tmem + sl * 64 + t * 32, ad + k * 2, bd + k * 2, idesc, k > 0);
        }
        umma_commit(&bars.empty[st]);
        umma_commit(&bars.tfull[sl]);
        ++it;
        return true;
      };
      for (int s = b1; s < e1 && ok; ++s) ok = step(ent[s / KB1 / G1].n, true);
      for (int s = b2; s < e2 && ok; ++s) {
        const int u = s / KB2, j = u / A;
        ok = step(ent[u - j * A].n, j * 256 + 128 < a.H);
      }
      umma_commit(&bars.drain);
      mbar_wait(&bars.drain, 0, never, limit);
    }
    __syncwarp();
  } else if (warp >= 4) {
    // ---- epilogue: 256 threads, thread = (tile of the step, weight row)
    const int et = tid - 128, tile = et >> 7, row = et & 127, ew = et >> 5;
    const uint32_t tlane = tmem + ((static_cast<uint32_t>(warp & 3) * 32u) << 16) + tile * 32;
    const int RS = pairs;  // rows of the scale arrays

    // this CTA's share of the activations: (token, 128-channel group) a warp
    for (int i = cta * 8 + ew; i < a.M * KB1; i += ctas * 8) {
      const int t = i / KB1, g = i - t * KB1;
      const int k = g * 128 + lane * 4;
      uint2 v = make_uint2(0, 0);
      if (k < a.H)  // H is a multiple of 16
        v = __ldg(reinterpret_cast<const uint2 *>(a.x + t * a.ldx + k));
      const float f[4] = {bf16_lo(v.x), bf16_hi(v.x), bf16_lo(v.y), bf16_hi(v.y)};
      float m = fmaxf(fmaxf(fabsf(f[0]), fabsf(f[1])), fmaxf(fabsf(f[2]), fabsf(f[3])));
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
      const float s = __fmul_rn(fmaxf(m, kFloor), kInv448);
      const uint32_t lo = __nv_cvt_float2_to_fp8x2(
          make_float2(__fdiv_rn(f[0], s), __fdiv_rn(f[1], s)), __NV_SATFINITE, __NV_E4M3);
      const uint32_t hi = __nv_cvt_float2_to_fp8x2(
          make_float2(__fdiv_rn(f[2], s), __fdiv_rn(f[3], s)), __NV_SATFINITE, __NV_E4M3);
      const uint32_t code = (lo & 0xFFFFu) | (hi << 16);
      for (int c = 0; c < a.topk; ++c) {
        if (ids[t * a.topk + c] < 0) continue;
        const int r = row_of[t * a.topk + c];
        *reinterpret_cast<uint32_t *>(a.xq + static_cast<int64_t>(r) * KB1 * 128 + k) = code;
        if (lane == 0) a.xs[static_cast<int64_t>(g) * RS + r] = s;
      }
    }
    __threadfence();
    fence_proxy_async_all();
    named_bar_sync(1, kEpi);
    if (et == 0) red_release_gpu(all_quant, 1);

    int it = 0;
    float acc[NT];
    // acc[n] = sum over K blocks [kb0, kb1) of a unit: partial sums from TMEM
    // times the weight block's scale (wscale[kb]) and token n's (xscale[kb * RS + n])
    auto sum_blocks = [&](int n, int kb0, int kb1, const float *wscale, const float *xscale,
                          bool on) {
#pragma unroll
      for (int i = 0; i < NT; ++i) acc[i] = 0.0f;
      float sx[4], nx[4], sw = 0.0f;
      auto fetch = [&](int kb) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          nx[i] = kb + i < kb1 && lane < n ? __ldcg(xscale + static_cast<int64_t>(kb + i) * RS + lane)
                                           : 0.0f;
      };
      fetch(kb0);
      for (int kb = kb0; kb < kb1; kb += 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) sx[i] = nx[i];
        if (((kb - kb0) & 31) == 0)
          sw = on && kb + lane < kb1 ? __ldg(wscale + kb + lane) : 0.0f;
        fetch(kb + 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (kb + i >= kb1) break;
          const int sl = it % kSlots;
          mbar_wait(&bars.tfull[sl], (it / kSlots) & 1, abort, limit);
          ++it;
          tc_fence_after();
          uint32_t v[NT];
          if (on) {
            tmem_ld16(tlane + sl * 64, v);
            if (NT > 16 && n > 16) tmem_ld16(tlane + sl * 64 + 16, v + (NT > 16 ? 16 : 0));
            tmem_ld_wait();
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars.tempty[sl]);
          if (!on) continue;
          const float w = __shfl_sync(0xFFFFFFFFu, sw, (kb + i - kb0) & 31);
#pragma unroll
          for (int c = 0; c < NT; ++c) {
            if (NT > 16 && c >= 16 && n <= 16) break;
            acc[c] = fmaf(__uint_as_float(v[c]),
                          __fmul_rn(w, __shfl_sync(0xFFFFFFFFu, sx[i], c)), acc[c]);
          }
        }
      }
    };

    // ---- first product
    if (b1 < e1) {
      wait_count(all_quant, ctas, abort, limit);
      __syncwarp();
    }
    for (int s = b1; s < e1;) {
      const int u = s / KB1, kb0 = s - u * KB1, kb1 = min(KB1, kb0 + e1 - s);
      const int ei = u / G1, g = u - ei * G1;
      const Entry en = ent[ei];
      sum_blocks(en.n, kb0, kb1,
                 a.s13 + (static_cast<int64_t>(en.e) * 2 * G1 + tile * G1 + g) * KB1,
                 a.xs + en.row, true);
      bool whole = true;
      if (kb1 - kb0 != KB1) {  // the sum is cut: publish this CTA's part
        const int c0 = owner_of(u * KB1, S1, P1), c1 = owner_of(u * KB1 + KB1 - 1, S1, P1);
        const int slot = u == b1 / KB1 ? 0 : 1;
        float *dst = a.part1 + ((static_cast<int64_t>(cta) * 2 + slot) * 2 + tile) * NT * 128 + row;
#pragma unroll
        for (int n = 0; n < NT; ++n)
          if (n < en.n) __stcg(dst + n * 128, acc[n]);
        __threadfence();
        named_bar_sync(1, kEpi);
        if (et == 0)
          bars.flag = atom_add_acq_rel_gpu(&unit_cnt[u], 1) == static_cast<uint32_t>(c1 - c0);
        named_bar_sync(1, kEpi);
        whole = bars.flag != 0;
        if (whole) {
          __threadfence();
#pragma unroll
          for (int n = 0; n < NT; ++n) acc[n] = 0.0f;
          for (int c = c0; c <= c1; ++c) {
            const int sl = u == run_begin(c, S1, P1) / KB1 ? 0 : 1;
            const float *src =
                a.part1 + ((static_cast<int64_t>(c) * 2 + sl) * 2 + tile) * NT * 128 + row;
#pragma unroll
            for (int n = 0; n < NT; ++n)
              if (n < en.n) acc[n] += __ldcg(src + n * 128);
          }
        }
      }
      if (whole) {
        float *hx = ysum;  // [NT][128]
        if (tile == 0) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
            if (n < en.n) hx[n * 128 + row] = acc[n];
        }
        named_bar_sync(1, kEpi);
        if (tile == 1) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
            if (n < en.n) {
              const float gate = hx[n * 128 + row];
              hx[n * 128 + row] = gate / (1.0f + expf(-gate)) * acc[n];
            }
        }
        named_bar_sync(1, kEpi);
        for (int n = ew; n < en.n; n += 8) {
          const float4 h = *reinterpret_cast<const float4 *>(hx + n * 128 + lane * 4);
          float m = fmaxf(fmaxf(fabsf(h.x), fabsf(h.y)), fmaxf(fabsf(h.z), fabsf(h.w)));
#pragma unroll
          for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
          const float sc = __fmul_rn(fmaxf(m, kFloor), kInv448);
          const uint32_t lo = __nv_cvt_float2_to_fp8x2(
              make_float2(__fdiv_rn(h.x, sc), __fdiv_rn(h.y, sc)), __NV_SATFINITE, __NV_E4M3);
          const uint32_t hi = __nv_cvt_float2_to_fp8x2(
              make_float2(__fdiv_rn(h.z, sc), __fdiv_rn(h.w, sc)), __NV_SATFINITE, __NV_E4M3);
          *reinterpret_cast<uint32_t *>(a.hq + static_cast<int64_t>(en.row + n) * a.I + g * 128 +
                                        lane * 4) = (lo & 0xFFFFu) | (hi << 16);
          if (lane == 0) a.hs[static_cast<int64_t>(g) * RS + en.row + n] = sc;
        }
        __threadfence();
        fence_proxy_async_all();
        named_bar_sync(1, kEpi);
        if (et == 0) red_release_gpu(&ready[ei], 1);
      }
      s += kb1 - kb0;
    }

    // ---- second product: ysum[token][256] of the output tile being summed;
    // a thread touches its own column of it alone
    const int per_tile = A * KB2;
    int head = -1, tail = -1;  // output tiles this CTA shares with others
    named_bar_sync(1, kEpi);   // the hidden rows' buffer is free
    for (int s = b2; s < e2;) {
      const int j = s / per_tile;
      const int s_end = min(e2, (j + 1) * per_tile);
      const bool mine = s == j * per_tile && s_end == (j + 1) * per_tile;
      const int s_first = s;
      const int col = j * 256 + et;
      const bool on = j * 256 + tile * 128 < a.H;
      for (int t = 0; t < a.M; ++t) ysum[t * 256 + et] = 0.0f;
      while (s < s_end) {
        const int u = s / KB2, kb0 = s - u * KB2, kb1 = min(KB2, kb0 + s_end - s);
        const int ei = u - j * A;
        const Entry en = ent[ei];
        wait_count(&ready[ei], G1, abort, limit);
        __syncwarp();
        sum_blocks(en.n, kb0, kb1,
                   a.s2 + (static_cast<int64_t>(en.e) * ((a.H + 127) / 128) + 2 * j + tile) * KB2,
                   a.hs + en.row, on);
#pragma unroll
        for (int n = 0; n < NT; ++n)
          if (n < en.n) {
            const int p = pair_of[en.row + n];
            float *at = ysum + (p / a.topk) * 256 + et;
            *at = fmaf(wgt[p], acc[n], *at);
          }
        s += kb1 - kb0;
      }
      if (mine) {
        if (col < a.H)
          for (int t = 0; t < a.M; ++t)
            a.y[static_cast<int64_t>(t) * a.H + col] = bf16_bits(ysum[t * 256 + et]);
      } else {
        const int slot = s_first == b2 ? 0 : 1;
        if (slot == 0) head = j;
        else tail = j;
        float *dst = a.part2 + (static_cast<int64_t>(cta) * 2 + slot) * a.M * 256 + et;
        for (int t = 0; t < a.M; ++t) __stcg(dst + t * 256, ysum[t * 256 + et]);
        __threadfence();
        named_bar_sync(1, kEpi);
        if (et == 0) red_release_gpu(&tile_cnt[j], 1);
      }
    }
    // shared output tiles: each of the tile's CTAs joins its share of the tokens
    for (int i = 0; i < 2; ++i) {
      const int j = i == 0 ? head : tail;
      if (j < 0) continue;
      const int c0 = owner_of(j * per_tile, S2, P2);
      const int c1 = owner_of((j + 1) * per_tile - 1, S2, P2);
      wait_count(&tile_cnt[j], c1 - c0 + 1, abort, limit);
      __syncwarp();
      const int col = j * 256 + et;
      for (int t = cta - c0; t < a.M; t += c1 - c0 + 1) {
        float v = 0.0f;
        for (int c = c0; c <= c1; ++c) {
          const int sl = run_begin(c, S2, P2) / per_tile == j ? 0 : 1;
          v += __ldcg(a.part2 + (static_cast<int64_t>(c) * 2 + sl) * a.M * 256 + t * 256 + et);
        }
        if (col < a.H) a.y[static_cast<int64_t>(t) * a.H + col] = bf16_bits(v);
      }
    }
    if (A == 0)  // no token chose an expert
      for (int64_t i = cta * kEpi + et; i < static_cast<int64_t>(a.M) * a.H; i += ctas * kEpi)
        a.y[i] = 0;
  }

  __syncthreads();
  if (tid == 0) {
    if (*abort) atomicMax(a.status, kStatusTimeout);
    bars.flag = atom_add_acq_rel_gpu(done, 1) == static_cast<uint32_t>(ctas - 1);
  }
  if (warp == 1) tmem_dealloc(tmem, 512);
  __syncthreads();
  if (bars.flag)  // the last CTA leaves the counters as it found them
    for (int i = tid; i < a.sync_words; i += kMoeThreads) a.sync[i] = 0;
}

int tokens_per_entry(int64_t M) { return M <= 16 ? 16 : 32; }

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

struct MoeLayout {
  size_t sync, xq, xs, hq, hs, part1, part2, total;
  int max_entries;
  int sync_words;
};

// Workspace: status word | counters | codes and scales of x and h, a row for
// each (token, choice) pair | partial sums of both products, two for each CTA
MoeLayout moe_layout(int64_t M, int64_t E, int64_t H, int64_t I, int64_t topk, int num_sms) {
  MoeLayout l;
  const int64_t P = M * topk, NT = tokens_per_entry(M);
  const int64_t KB1 = (H + 127) / 128, G1 = I / 128, J = (H + 255) / 256;
  l.max_entries = static_cast<int>((E < P ? E : P) + P / NT);
  l.sync_words = static_cast<int>(32 + J + l.max_entries * (1 + G1));
  size_t at = 256;
  auto take = [&](int64_t bytes) {
    const size_t here = at;
    at += up256(static_cast<size_t>(bytes));
    return here;
  };
  l.sync = take(l.sync_words * 4);
  l.xq = take(P * KB1 * 128);
  l.xs = take(P * KB1 * 4);
  l.hq = take(P * I);
  l.hs = take(P * G1 * 4);
  l.part1 = take(static_cast<int64_t>(num_sms) * 2 * 2 * NT * 128 * 4);
  l.part2 = take(static_cast<int64_t>(num_sms) * 2 * M * 256 * 4);
  l.total = at;
  return l;
}

}  // namespace

size_t moe_workspace(int64_t M, int64_t E, int64_t H, int64_t I, int64_t topk) {
  return moe_layout(M, E, H, I, topk, kMoeMaxCtas).total;
}

cudaError_t launch_moe_layer(MoeArgs a, const void *w13, const void *w2, void *ws,
                             const DeviceInfo &dev, cudaStream_t st) {
  const int ctas = dev.num_sms < kMoeMaxCtas ? dev.num_sms : kMoeMaxCtas;
  const MoeLayout l = moe_layout(a.M, a.E, a.H, a.I, a.topk, kMoeMaxCtas);
  uint8_t *base = static_cast<uint8_t *>(ws);
  a.status = reinterpret_cast<uint32_t *>(base);
  a.sync = reinterpret_cast<uint32_t *>(base + l.sync);
  a.xq = base + l.xq;
  a.xs = reinterpret_cast<float *>(base + l.xs);
  a.hq = base + l.hq;
  a.hs = reinterpret_cast<float *>(base + l.hs);
  a.part1 = reinterpret_cast<float *>(base + l.part1);
  a.part2 = reinterpret_cast<float *>(base + l.part2);
  a.max_entries = l.max_entries;
  a.sync_words = l.sync_words;
  const int64_t P = static_cast<int64_t>(a.M) * a.topk, KB1 = (a.H + 127) / 128;
  const int NT = tokens_per_entry(a.M);
  const size_t ysum = static_cast<size_t>(a.M * 256 > NT * 128 ? a.M * 256 : NT * 128) * 4;
  const size_t fixed = 1024 + ysum + P * 4 + static_cast<size_t>(l.max_entries) * sizeof(Entry) +
                       static_cast<size_t>(a.E) * 4 + P * 6;
  const size_t stage = 2 * kTileBytes + NT * 128;
  const size_t room = dev.max_smem_optin - 1024;  // the static part
  a.stages = static_cast<int>((room - fixed) / stage);
  if (a.stages > kMaxRing) a.stages = kMaxRing;
  const size_t smem = fixed + a.stages * stage;

  CUtensorMap m13, m2, mx, mh;
  if (!make_kmajor_map(&m13, w13, static_cast<int64_t>(a.E) * 2 * a.I, a.H, 128) ||
      !make_kmajor_map(&m2, w2, static_cast<int64_t>(a.E) * a.H, a.I, 128) ||
      !make_kmajor_map(&mx, a.xq, P, KB1 * 128, 16) || !make_kmajor_map(&mh, a.hq, P, a.I, 16))
    return cudaErrorInvalidValue;
  auto run = [&](auto kern) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeCooperative;  // every CTA resident, or an error
    attr[0].val.cooperative = 1;
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kMoeThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, m13, m2, mx, mh, a);
  };
  return NT == 16 ? run(moe_layer_kernel<16>) : run(moe_layer_kernel<32>);
}

}  // namespace fp8bq
