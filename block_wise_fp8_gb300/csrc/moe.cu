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
// the steps that depend on one another.  Measured: 209 us for 16 tokens that reach 30
// of 32 experts of 7168 x 2048 (1.31 GB, 6.25 TB/s), 343 us for 61 tokens over 125 of
// 128 of 4096 x 1408 (6.3 TB/s), 70 us for one token of 8 of the former (5.0 TB/s: the
// launch, the way to the first weights, the hand-over of h and the last sums take
// about 15 us), 22 us for one of 4 of 2048 x 768, which is those alone.
// So the layer is one persistent kernel, one CTA an SM (a cooperative launch,
// since CTAs wait on one another), and its weight copies never wait for
// activations: a warp streams the weight tiles of both products, in order,
// through a ring in shared memory, while a second warp adds the activation tiles
// to the same stages once the CTAs that produce them have published them.  Across
// each dependency (quantised x, the experts' h) the ring fills with weights
// instead of draining.
//
// Both products are cut into units -- 128 hidden columns of an expert (its gate
// and up rows), or two 128-row tiles of its output -- and a unit's sum over K
// into runs of a few steps; a step is two 128 x 128 weight tiles that share an
// activation tile.  CTAs take the runs in turn: all of the first product, expert
// by expert, then the second's in the same order, so that the first experts' h
// is long finished when the second product begins.  (Dealt equally in advance,
// the slowest SMs finished up to a third later than the rest: 276 against 240 us
// for 16 tokens of 32 experts of 7168 x 2048.)  The epilogue warps leave a run's
// sums in the workspace and go on; they wait for nobody but the tensor core.
// Two warps of a CTA that the unit names add the runs' sums of the first product
// and make h of them; those of the second are added when all is done, each CTA
// taking its share of the outputs.  The runs' bounds and every order of addition
// follow from the sizes and the routing alone, so results repeat bit for bit
// whoever took which run.
//
// The tensor core sees the weights as the 128 rows of A and up to NT tokens as
// the columns of B (tcgen05.mma, M = 128).  In the first product the columns
// are all tokens, whoever chose the expert: x then needs no order by expert
// and is quantised while the routing is still going on.  The epilogue reads the
// chosen tokens' columns alone, one by one: 0.8 us a step where an expert has 15
// tokens and more, which small experts do not hide.  In the second they are the entry's hidden
// rows.  Tokens of one expert beyond NT form a further entry that reads the
// weights again, from L2.
//
// Routing is computed by every CTA for itself: at these sizes that is cheaper
// than one CTA's result handed to the others.
#include "common.cuh"
#include "ptx.cuh"
#include "quant_math.cuh"

namespace fp8bq {
namespace {

// Warps: 0 weight copies, 2 activation copies, 1 and 3 MMA issuers, 4 to 11 the
// epilogue, 12 signals, 13 scales, 14 and 15 finish h.  One MMA instruction of so
// few columns takes its issuer about 0.06 us: a single issuer set the pace (0.75
// us for a step's eight, HBM half idle), so two take the stages in turn.
constexpr int kMoeThreads = 512;
constexpr int kIssuers = 2;
constexpr int kSignals = 4;
constexpr int kEpi = 256;
constexpr int kEpiWarps = 8;
constexpr int kTileBytes = 128 * 128;
constexpr int kMaxRing = 4;
constexpr int kRunQueue = 4;
// The codes never leave the layer, so the scale is a product with the binary32
// reciprocal, not the quantisers' division.  It differs from theirs by one binary32
// step in 57 % of the groups of normal BF16 rows, which moves the codes of
// quotients that are exact ties (0.09 % of them) to the other, equally near, one.
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

// Asynchronous 4-byte copy global -> shared; an arrival on `bar` once all of this
// thread's copies so far have landed (counted in the barrier's init count).
__device__ __forceinline__ void copy4_async(float *dst, const float *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void arrive_when_copied(uint64_t *bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void copies_landed() { asm volatile("cp.async.wait_all;" ::: "memory"); }

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

__device__ __forceinline__ float sigmoid(float l) { return __frcp_rn(1.0f + expf(-l)); }

// Group-128 quantisation by a warp, four values a lane: codes and scale.
__device__ __forceinline__ uint32_t quant4(const float (&f)[4], float *scale) {
  float m = fmaxf(fmaxf(fabsf(f[0]), fabsf(f[1])), fmaxf(fabsf(f[2]), fabsf(f[3])));
  m = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(m)));  // m >= 0
  const float s = __fmul_rn(fmaxf(m, kFloor), kInv448);
  // RN(x / s) without a division: one corrected step from x RN(1 / s)
  // (Markstein's theorem); where the remainder underflows the code is 0 anyway
  const float r = __frcp_rn(s);
  float q[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    q[i] = __fmul_rn(f[i], r);
    q[i] = __fmaf_rn(__fmaf_rn(-s, q[i], f[i]), r, q[i]);
  }
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(q[0], q[1]), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(q[2], q[3]), __NV_SATFINITE, __NV_E4M3);
  *scale = s;
  return (lo & 0xFFFFu) | (hi << 16);
}

// 32 lanes x 32 bit of one column.
__device__ __forceinline__ void tmem_ld1(uint32_t taddr, uint32_t &r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r) : "r"(taddr));
}

// Expert entry: expert, first row of its tokens in the order of the hidden rows,
// tokens (at most NT)
struct Entry {
  int e, row, n;
};

// Runs a unit of KB steps is cut into: runs of about 8 steps, or shorter ones
// where all units together give a CTA less than 12 steps; `most` bounds the
// workspace.
__device__ __forceinline__ int runs_of(int KB, int units, int ctas, int most) {
  const int each = (units * KB + ctas - 1) / ctas;
  return min(most, (KB + (each < 12 ? max(each, 1) : 8) - 1) / (each < 12 ? max(each, 1) : 8));
}

// What the weight warp hands to the others: a run of one of the products
// (0: no more), K blocks kb .. kb + steps - 1 of entry ei's unit `sub`, whose
// sums go to plane `plane`.
struct Run {
  int product, ei, sub, plane, kb, steps;
};

struct MoeBars {
  uint64_t full_w[kMaxRing], full_b[kMaxRing], empty[kMaxRing];
  uint64_t tfull[kMaxRing], tempty[kMaxRing];
  uint64_t run_full[kRunQueue], run_empty[kRunQueue];
  uint64_t sig[kSignals], sig_free[kSignals];
  uint64_t drain;
  Run run[kRunQueue];
  uint32_t tmem;
  uint32_t abort, never;  // never stays 0
  uint32_t last;
  int entries;
};

// ---------------------------------------------------------------- routing

// Order-preserving keys of binary32 numbers; 0 stands for "not to be chosen"
// (-inf, NaN), +inf counts as the largest finite number, -0 as 0.
__device__ __forceinline__ uint32_t key_of(float l) {
  if (!(l > -INFINITY)) return 0;
  const uint32_t u = __float_as_uint(fminf(l, 3.402823466e38f) + 0.0f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}

// The choice of tokens t0, t0 + step, ... by one warp, for up to 32 R experts:
// ids into id[t * kMoeMaxTopk ..], weights into w[t * kMoeMaxTopk ..].  Lane i holds the
// keys of experts i, i + 32, ...; a chosen key becomes 0, and lane k keeps the
// k-th choice, so that the weights are computed once, side by side.
template <int R>
__device__ void route_tokens(const MoeArgs &a, int t0, int step, short *id, float *w) {
  const int lane = threadIdx.x & 31;
  float l[R];
  auto fetch = [&](int t) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int e = r * 32 + lane;
      l[r] = t < a.M && e < a.E ? __ldg(a.logits + static_cast<int64_t>(t) * a.E + e) : -INFINITY;
    }
  };
  fetch(t0);
  for (int t = t0; t < a.M; t += step) {
    const float *row = a.logits + static_cast<int64_t>(t) * a.E;
    uint32_t key[R];
#pragma unroll
    for (int r = 0; r < R; ++r) key[r] = key_of(l[r]);
    fetch(t + step);
    float denom = 1.0f;
    uint32_t top = 0;
    if (a.score == 0) {
#pragma unroll
      for (int r = 0; r < R; ++r) top = max(top, key[r]);
      top = __reduce_max_sync(0xFFFFFFFFu, top);
      if (!a.renorm) {  // renormalised, the sum over all experts cancels
        float s = 0.0f;
#pragma unroll
        for (int r = 0; r < R; ++r)
          if (key[r]) s += expf(value_of(key[r]) - value_of(top));
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
        denom = s;
      }
    }
    if (a.bias) {  // chosen by sigmoid + bias
#pragma unroll
      for (int r = 0; r < R; ++r)
        if (key[r]) key[r] = key_of(sigmoid(value_of(key[r])) + __ldg(a.bias + r * 32 + lane));
    }
    uint32_t got = 0;  // lane k: key and index of choice k
    int got_at = -1;
    for (int k = 0; k < a.topk; ++k) {
      uint32_t m = 0;
#pragma unroll
      for (int r = 0; r < R; ++r) m = max(m, key[r]);
      const uint32_t best = __reduce_max_sync(0xFFFFFFFFu, m);
      if (best == 0) break;
      int at = 1 << 20;
#pragma unroll
      for (int r = R - 1; r >= 0; --r)
        if (key[r] == best) at = r * 32 + lane;
      at = __reduce_min_sync(0xFFFFFFFFu, at);
      if (a.bias) {
        // Keys this close may be ordered by binary32 rounding (a few 2^-24 of
        // a sigmoid below 1 and of the sum): such a choice is made in 64 bits.
        // (A sum near the lowest number has no border below it: the difference is
        // -inf and its key 0, that of a taken, masked or missing expert.)
        const float v = value_of(best);
        const uint32_t near = max(key_of(v - (1e-6f + 4e-7f * fabsf(v))), 1u);
        int close = 0;
#pragma unroll
        for (int r = 0; r < R; ++r) close += key[r] >= near ? 1 : 0;
        if (__reduce_add_sync(0xFFFFFFFFu, close) > 1) {
          double bd = -1e300;
          int bat = 1 << 20;
#pragma unroll
          for (int r = 0; r < R; ++r)
            if (key[r] >= near) {
              const int e = r * 32 + lane;
              const double x = fminf(__ldg(row + e), 3.402823466e38f);
              const double d = 1.0 / (1.0 + exp(-x)) + static_cast<double>(__ldg(a.bias + e));
              if (d > bd) bd = d, bat = e;
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
      if (lane == k) got = best, got_at = at;
#pragma unroll
      for (int r = 0; r < R; ++r)
        if (lane + r * 32 == at) key[r] = 0;
    }
    float x = 0.0f, v = 0.0f;
    if (got_at >= 0) {
      x = a.bias ? fminf(__ldg(row + got_at), 3.402823466e38f) : value_of(got);
      v = a.score == 0 ? expf(x - value_of(top)) / denom : sigmoid(x);
    }
    // Sigmoids near binary32's smallest numbers (e^-87) and below have shares all
    // the same; they are taken in 64 bits, whose own end is at e^-709.
    if (a.renorm && a.score != 0 && __any_sync(0xFFFFFFFFu, x < -80.0f)) {
      const double p = got_at >= 0 ? 1.0 / (1.0 + exp(-static_cast<double>(x))) : 0.0;
      double s = p;
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
      v = s > 0.0 ? static_cast<float>(p / s) : 0.0f;
    } else if (a.renorm) {
      float s = v;
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
      v = s > 0.0f ? v / s : 0.0f;
    }
    if (lane < kMoeMaxTopk) {  // got_at stays -1 from topk on
      id[t * kMoeMaxTopk + lane] = static_cast<short>(got_at);
      w[t * kMoeMaxTopk + lane] = v * a.scale;
    }
  }
}

// ---------------------------------------------------------------- the kernel

// One hidden row's 128 columns of group g by a warp: h = silu(gate) * up, codes
// and scale.
__device__ void hidden_row(const MoeArgs &a, float4 gate, float4 up, int row, int g, float *scale) {
  const int lane = threadIdx.x & 31;
  const float f[4] = {gate.x * sigmoid(gate.x) * up.x, gate.y * sigmoid(gate.y) * up.y,
                      gate.z * sigmoid(gate.z) * up.z, gate.w * sigmoid(gate.w) * up.w};
  float sc;
  const uint32_t code = quant4(f, &sc);
  *reinterpret_cast<uint32_t *>(a.hq + static_cast<int64_t>(row) * a.I + g * 128 + lane * 4) = code;
  if (lane == 0) *scale = sc;
}

template <int NT>
struct MoeCfg {
  static constexpr int kTokens = NT == 16 ? 16 : kMoeMaxTokens;
  static constexpr int kStage = 2 * kTileBytes + kTokens * 128;
  static constexpr int kCols = kTokens;              // TMEM columns of one partial tile
  // Four stages (64 KB and more of weights in flight an SM): with six the copies
  // queue for 8 us and more in HBM, which delays everything else (67.6 against
  // 73.7 us at one token of 8 experts of 7168 x 2048), with three HBM idles (74).
  static constexpr int kMaxStages = kMaxRing;  // a stage has a TMEM buffer of two tiles
  static constexpr int kTmemCols = kMaxStages * 2 * kCols;
};

template <int NT>
__global__ void __launch_bounds__(kMoeThreads, 1)
    moe_layer_kernel(const __grid_constant__ CUtensorMap map13,
                     const __grid_constant__ CUtensorMap map2,
                     const __grid_constant__ CUtensorMap mapx,
                     const __grid_constant__ CUtensorMap maph, const MoeArgs a) {
  using C = MoeCfg<NT>;
  constexpr int kStage = C::kStage, kCols = C::kCols;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ MoeBars bars;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int cta = blockIdx.x, ctas = gridDim.x;
  const uint64_t limit = a.wait_limit_ns;
  volatile uint32_t *abort = &bars.abort;
  volatile uint32_t *never = &bars.never;
  const int pairs = a.M * a.topk;
  const int KB1 = (a.H + 127) / 128, G1 = a.I / 128, KB2 = G1;
  const int J = (a.H + 255) / 256;

  uint8_t *ring = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  float *scl = reinterpret_cast<float *>(ring + a.stages * kStage);  // [stages][NT + 4] scales
  float *wgt = scl + a.stages * (NT + 4);                    // [M][16]: weight by choice
  float *wrow = wgt + a.M * kMoeMaxTopk;                    // [pairs]: by hidden row
  Entry *ent = reinterpret_cast<Entry *>(wrow + pairs);     // [max_entries]
  uint32_t *mask = reinterpret_cast<uint32_t *>(ent + a.max_entries);  // [E][2]: tokens' bits
  int *first = reinterpret_cast<int *>(mask + 2 * a.E);     // [E]: first hidden row
  short *ids = reinterpret_cast<short *>(first + a.E);      // [M][16], -1: none
  short *row_of = ids + a.M * kMoeMaxTopk;                  // [M][16]: hidden row, -1: none
  short *tok = row_of + a.M * kMoeMaxTopk;                  // [pairs]: token of a hidden row

  uint32_t *const all_quant = a.sync;       // CTAs whose share of x is quantised
  uint32_t *const all_done = a.sync + 1;    // CTAs without a run left
  uint32_t *const leaving = a.sync + 2;
  uint32_t *const claim = a.sync + 3;       // runs taken, past the first round
  uint32_t *const units_done = a.sync + 4;  // hidden groups published,
  uint32_t *const ready = a.sync + 32;      // [entries]: by entry
  uint32_t *const unit_cnt = ready + a.max_entries;  // [entries * G1]: runs done
  const uint32_t quant_ctas = min(ctas, a.M * KB1);

  if (tid == 0) {
    for (int i = 0; i < a.stages; ++i) {
      mbar_init(&bars.full_w[i], 1);
      mbar_init(&bars.full_b[i], 1);
      mbar_init(&bars.empty[i], 1);
    }
    for (int i = 0; i < a.stages; ++i) {
      mbar_init(&bars.tfull[i], 1 + 32);  // the products, and the scale warp's lanes
      mbar_init(&bars.tempty[i], kEpiWarps);
    }
    for (int i = 0; i < kRunQueue; ++i) {
      mbar_init(&bars.run_full[i], 1);
      mbar_init(&bars.run_empty[i], 3 + kIssuers + kEpiWarps);
    }
    for (int i = 0; i < kSignals; ++i) {
      mbar_init(&bars.sig[i], kEpiWarps);
      mbar_init(&bars.sig_free[i], 1);
    }
    mbar_init(&bars.drain, kIssuers);
    bars.abort = 0;
    bars.never = 0;
    fence_mbar_init();
    tma_prefetch_desc(&map13);
    tma_prefetch_desc(&map2);
    tma_prefetch_desc(&mapx);
    tma_prefetch_desc(&maph);
  }
  if (warp == 1) {
    tmem_alloc(&bars.tmem, C::kTmemCols);
    tmem_relinquish();
  }
  for (int e = tid; e < 2 * a.E; e += kMoeThreads) mask[e] = 0;

  // ---- this CTA's share of the activations: a (token, 128-channel group) a
  // warp, dealt to the CTAs first
  if (warp >= 4 && warp < 12) {
    for (int i = (warp - 4) * ctas + cta; i < a.M * KB1; i += ctas * 8) {
      const int t = i / KB1, g = i - t * KB1;
      const int k = g * 128 + lane * 4;
      uint2 v = make_uint2(0, 0);
      if (k < a.H)  // H is a multiple of 16
        v = __ldg(reinterpret_cast<const uint2 *>(a.x + t * a.ldx + k));
      const float f[4] = {bf16_lo(v.x), bf16_hi(v.x), bf16_lo(v.y), bf16_hi(v.y)};
      float s;
      const uint32_t code = quant4(f, &s);
      *reinterpret_cast<uint32_t *>(a.xq + static_cast<int64_t>(t) * KB1 * 128 + k) = code;
      if (lane == 0) a.xs[g * a.M + t] = s;
    }
    fence_proxy_async_all();  // the codes are read by TMA
    named_bar_sync(1, kEpi);
    if (tid == 128 && cta < static_cast<int>(quant_ctas)) red_release_gpu(all_quant, 1);
  }

  // ---- routing, by every CTA
  if (a.logits) {
    if (a.E <= 128) route_tokens<4>(a, warp, kMoeThreads / 32, ids, wgt);
    else if (a.E <= 256) route_tokens<8>(a, warp, kMoeThreads / 32, ids, wgt);
    else route_tokens<16>(a, warp, kMoeThreads / 32, ids, wgt);
  } else {
    for (int p = tid; p < a.M * kMoeMaxTopk; p += kMoeThreads) {
      const int k = p % kMoeMaxTopk, at = p / kMoeMaxTopk * a.topk + k;
      const int e = k < a.topk ? __ldg(a.ids_in + at) : -1;
      ids[p] = e >= 0 && e < a.E ? static_cast<short>(e) : -1;
      wgt[p] = k < a.topk ? __ldg(a.w_in + at) : 0.0f;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // each expert's tokens as a bit mask, the same in whatever order it is made
  for (int p = tid; p < a.M * kMoeMaxTopk; p += kMoeThreads) {
    const int e = ids[p], t = p / kMoeMaxTopk;
    if (e >= 0) atomicOr(&mask[2 * e + (t >> 5)], 1u << (t & 31));
  }
  __syncthreads();
  if (warp == 0) {
    // entries and first hidden rows: each lane takes neighbouring experts
    const int per = (a.E + 31) / 32;
    int rows = 0, n_ent = 0;
    for (int i = 0; i < per; ++i) {
      const int e = lane * per + i;
      const int n = e < a.E ? __popc(mask[2 * e]) + __popc(mask[2 * e + 1]) : 0;
      rows += n, n_ent += (n + NT - 1) / NT;
    }
    int rr = rows, ee = n_ent;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int v = __shfl_up_sync(0xFFFFFFFFu, rr, d);
      const int u = __shfl_up_sync(0xFFFFFFFFu, ee, d);
      if (lane >= d) rr += v, ee += u;
    }
    if (lane == 31) bars.entries = ee;
    rr -= rows, ee -= n_ent;
    for (int i = 0; i < per; ++i) {
      const int e = lane * per + i;
      if (e >= a.E) break;
      const int n = __popc(mask[2 * e]) + __popc(mask[2 * e + 1]);
      first[e] = rr;
      for (int k = 0; k < n; k += NT) ent[ee++] = Entry{e, rr + k, min(NT, n - k)};
      rr += n;
    }
  }
  __syncthreads();
  for (int p = tid; p < a.M * kMoeMaxTopk; p += kMoeThreads) {
    const int e = ids[p], t = p / kMoeMaxTopk, k = p % kMoeMaxTopk;
    row_of[p] = -1;
    if (e < 0) continue;
    // a token that names an expert twice has one row, with both weights
    float w = wgt[p];
    bool again = false;
#pragma unroll 1
    for (int i = 1; i < a.topk; ++i) {
      const int o = k + i < a.topk ? p + i : p + i - a.topk;
      if (ids[o] != e) continue;
      again |= o < p;
      w += wgt[o];
    }
    if (again) continue;
    const uint32_t lo = mask[2 * e], hi = mask[2 * e + 1], below = (1u << (t & 31)) - 1u;
    const int r = first[e] + (t < 32 ? __popc(lo & below) : __popc(lo) + __popc(hi & below));
    tok[r] = static_cast<short>(t);
    row_of[p] = static_cast<short>(r);
    wrow[r] = w;
  }
  __syncthreads();

  if (cta == 0 && warp >= 14)
    for (int p = tid - 14 * 32; p < pairs; p += 64) {
      const int at = p / a.topk * kMoeMaxTopk + p % a.topk;
      if (a.ids_out) a.ids_out[p] = ids[at];
      if (a.w_out) a.w_out[p] = wgt[at];
    }

  const int A = bars.entries;
  const int R1 = runs_of(KB1, A * G1, ctas, a.planes), R2 = runs_of(KB2, A * J, ctas, a.planes);
  // a plane holds one run of every sum, by hidden row (and a spare row)
  const int64_t plane1 = static_cast<int64_t>(pairs + 1) * 2 * a.I;
  const int64_t plane2 = static_cast<int64_t>(pairs) * a.H;
  const int all1 = A * G1 * R1, all_runs = all1 + A * J * R2;
  const uint32_t tmem = bars.tmem;

  if (warp == 0) {
    if (lane == 0) {  // ---- weight tiles
      int st = 0, ph = 1, it = 0;  // stage, the parity its release is waited with, steps issued
      int qi = 0, qph = 1;
      bool ok = true;
      auto hand = [&](Run r) {
        ok = mbar_wait(&bars.run_empty[qi], qph, abort, limit);
        if (!ok) return;
        bars.run[qi] = r;
        mbar_arrive(&bars.run_full[qi]);
        if (++qi == kRunQueue) qi = 0, qph ^= 1;
      };
      auto stage = [&](const CUtensorMap *map, int kb, int r0, int r1, bool two) {
        ok = mbar_wait(&bars.empty[st], ph, abort, limit);
        if (!ok) return;
        if (!(a.fault && cta == 0 && it == 0)) {  // fault injection: this stage's wait runs out
          uint8_t *dst = ring + st * kStage;
          mbar_arrive_expect_tx(&bars.full_w[st], two ? 2 * kTileBytes : kTileBytes);
          tma_load_2d(dst, map, &bars.full_w[st], kb * 128, r0);
          if (two) tma_load_2d(dst + kTileBytes, map, &bars.full_w[st], kb * 128, r1);
        }
        ++it;
        if (++st == a.stages) st = 0, ph ^= 1;
      };
      for (int pos = cta; pos < all_runs && ok;) {
        const int next = ctas + static_cast<int>(atomicAdd(claim, 1u));
        const bool one = pos < all1;
        const int KB = one ? KB1 : KB2, R = one ? R1 : R2, U = one ? G1 : J;
        const int q = one ? pos : pos - all1, u = q / R;
        Run run;
        run.product = one ? 1 : 2, run.plane = q - u * R;
        run.ei = u / U, run.sub = u - run.ei * U;
        run.kb = run.plane * KB / R, run.steps = (run.plane + 1) * KB / R - run.kb;
        hand(run);
        const int64_t e = ent[run.ei].e;
        const int nb2 = (a.H + 127) / 128;
        const float *sc = (one ? a.s13 + (e * 2 * G1 + run.sub) * KB1 : a.s2 + (e * nb2 + 2 * run.sub) * KB2) + run.kb;
        prefetch_l2(sc);
        if (one || run.sub * 2 + 1 < nb2) prefetch_l2(sc + (one ? G1 * KB1 : KB2));
        const int r = static_cast<int>(one ? e * 2 * a.I + run.sub * 128 : e * a.H + run.sub * 256);
        const CUtensorMap *map = one ? &map13 : &map2;
        for (int i = 0; i < run.steps && ok; ++i)
          stage(map, run.kb + i, r, one ? r + a.I : r + 128, one || run.sub * 256 + 128 < a.H);
        pos = next;
      }
      if (ok) hand(Run{0, 0, 0, 0, 0, 0});
      if (!ok)  // let the copies in flight land before this CTA's memory is given up
        for (int i = max(a.fault && cta == 0 ? 1 : 0, it - a.stages); i < it; ++i)
          mbar_wait(&bars.full_w[i % a.stages], (i / a.stages) & 1, never, limit);
    }
    __syncwarp();
  } else if (warp == 2) {
    if (lane == 0) {  // ---- activation tiles
      int st = 0, ph = 1, it = 0, qi = 0, qph = 0;
      bool ok = true, quantised = false, hidden = false;
      const int xboxes = (a.M + 15) / 16;  // every token's row: the epilogue picks columns
      while (ok) {
        ok = mbar_wait(&bars.run_full[qi], qph, abort, limit);
        if (!ok) break;
        const Run run = bars.run[qi];
        mbar_arrive(&bars.run_empty[qi]);
        if (++qi == kRunQueue) qi = 0, qph ^= 1;
        if (run.product == 0) break;
        const CUtensorMap *map = &mapx;
        int row = 0, boxes = xboxes;
        if (run.product == 1) {
          if (!quantised) {
            ok = quantised = wait_count(all_quant, quant_ctas, abort, limit);
            fence_proxy_async_all();
          }
        } else {
          if (!hidden) {
            hidden = ld_acquire_gpu(units_done) >= static_cast<uint32_t>(A * G1);
            if (!hidden) ok = wait_count(&ready[run.ei], G1, abort, limit);
            fence_proxy_async_all();
          }
          map = &maph, row = ent[run.ei].row, boxes = (ent[run.ei].n + 15) / 16;
        }
        for (int i = 0; i < run.steps && ok; ++i) {
          ok = mbar_wait(&bars.empty[st], ph, abort, limit);
          if (!ok) break;
          uint8_t *dst = ring + st * kStage + 2 * kTileBytes;
          mbar_arrive_expect_tx(&bars.full_b[st], boxes * 2048);
          for (int b = 0; b < boxes; ++b)
            tma_load_2d(dst + b * 2048, map, &bars.full_b[st], (run.kb + i) * 128, row + b * 16);
          ++it;
          if (++st == a.stages) st = 0, ph ^= 1;
        }
      }
      if (!ok)
        for (int i = max(0, it - a.stages); i < it; ++i)
          mbar_wait(&bars.full_b[i % a.stages], (i / a.stages) & 1, never, limit);
    }
    __syncwarp();
  } else if (warp == 1 || warp == 3) {
    if (lane == 0) {  // ---- MMAs
      // A stage, and the TMEM buffer of the same number, belong to one issuer:
      // a parity wait tells two phases apart, not three, so whoever waits for
      // a stage's phase must have seen the one before.
      const int st0 = warp >> 1;
      int st = st0, ph = 0, it = st0;  // this issuer's next step
      int it0 = 0, qi = 0, qph = 0;    // the run's first step
      bool ok = true;
      while (ok) {
        ok = mbar_wait(&bars.run_full[qi], qph, abort, limit);
        if (!ok) break;
        const Run run = bars.run[qi];
        mbar_arrive(&bars.run_empty[qi]);
        if (++qi == kRunQueue) qi = 0, qph ^= 1;
        if (run.product == 0) break;
        const int it1 = it0 + run.steps;
        const int n = run.product == 1 ? a.M : ent[run.ei].n;
        const bool two = run.product == 1 || run.sub * 256 + 128 < a.H;
        const uint32_t idesc = idesc_f8f6f4_e4m3(128, (n + 15) / 16 * 16);
        while (it < it1) {
          ok = mbar_wait(&bars.tempty[st], ph ^ 1, abort, limit) &&
               mbar_wait(&bars.full_w[st], ph, abort, limit) &&
               mbar_wait(&bars.full_b[st], ph, abort, limit);
          if (!ok) break;
          tc_fence_after();
          const uint32_t base = smem_u32(ring + st * kStage);
          const uint64_t bd = sdesc_kmajor_sw128(base + 2 * kTileBytes);
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (t == 1 && !two) break;
            const uint64_t ad = sdesc_kmajor_sw128(base + t * kTileBytes);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              umma_f8f6f4(tmem + (st * 2 + t) * kCols, ad + k * 2, bd + k * 2, idesc, k > 0);
          }
          umma_commit(&bars.empty[st]);
          umma_commit(&bars.tfull[st]);
          // on to this issuer's next stage: the steps between are the others'
          if (st + kIssuers < a.stages) st += kIssuers, it += kIssuers;
          else it += a.stages - st + st0, st = st0, ph ^= 1;
        }
        it0 = it1;
      }
      umma_commit(&bars.drain);
      mbar_wait(&bars.drain, 0, never, limit);
    }
    __syncwarp();
  } else if (warp == 12) {
    // ---- signals: a release at GPU scope takes microseconds while the weights
    // stream (3.5 us measured; the epilogue, which did it itself, fell behind
    // HBM), so this warp does it for the epilogue warps, a run of the first
    // product at a time, and once more when all runs are done
    if (lane == 0) {
      int qi = 0, qph = 0, sg = 0, sph = 0;
      bool more = true;
      while (more && mbar_wait(&bars.run_full[qi], qph, abort, limit)) {
        const Run run = bars.run[qi];
        mbar_arrive(&bars.run_empty[qi]);
        if (++qi == kRunQueue) qi = 0, qph ^= 1;
        more = run.product != 0;
        if (run.product == 2) continue;
        if (!mbar_wait(&bars.sig[sg], sph, abort, limit)) break;
        red_release_gpu(more ? &unit_cnt[run.ei * G1 + run.sub] : all_done, 1);
        mbar_arrive(&bars.sig_free[sg]);
        if (++sg == kSignals) sg = 0, sph ^= 1;
      }
    }
    __syncwarp();
  } else if (warp == 13) {
    // ---- scales: per step the rows' and the two weight blocks', copied
    // asynchronously into the stage's own place as soon as the epilogue has
    // left it, so that up to a ring's length of copies is in flight (loads
    // through registers were 3 us late where the weights streamed)
    int st = 0, ph = 1, qi = 0, qph = 0;
    bool quantised = false, hidden = false;
    const int nbs2 = (a.H + 127) / 128;
    while (__all_sync(0xFFFFFFFFu, mbar_wait(&bars.run_full[qi], qph, abort, limit))) {
      const Run run = bars.run[qi];
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.run_empty[qi]);
      if (++qi == kRunQueue) qi = 0, qph ^= 1;
      if (run.product == 0) break;
      const bool one = run.product == 1;
      if (one ? !quantised : !hidden) {
        if (one) {
          wait_count(all_quant, quant_ctas, abort, limit);
          quantised = true;
        } else {
          hidden = __all_sync(0xFFFFFFFFu,
                              ld_acquire_gpu(units_done) >= static_cast<uint32_t>(A * G1));
          if (!hidden) wait_count(&ready[run.ei], G1, abort, limit);
        }
        __syncwarp();
      }
      const Entry en = ent[run.ei];
      const int64_t e = en.e;
      const float *w0 =
          (one ? a.s13 + (e * 2 * G1 + run.sub) * KB1 : a.s2 + (e * nbs2 + 2 * run.sub) * KB2) + run.kb;
      const float *w1 = one ? w0 + G1 * KB1 : 2 * run.sub + 1 < nbs2 ? w0 + KB2 : w0;
      // an entry's scales of one block of h have a cache line of their own: these
      // copies pass through L1, which must not keep a line that is still written to
      const int xstride = one ? a.M : 32;
      const float *x = (one ? a.xs + (lane < en.n ? tok[en.row + lane] : 0)
                            : a.hs + run.ei * G1 * 32 + lane) + run.kb * xstride;
      for (int i = 0; i < run.steps; ++i) {
        mbar_wait(&bars.tempty[st], ph, abort, limit);
        __syncwarp();
        float *dst = scl + st * (NT + 4);
        if (lane < en.n) copy4_async(dst + lane, x);
        if (lane < 2) copy4_async(dst + NT + lane, lane ? w1 : w0);
        arrive_when_copied(&bars.tfull[st]);
        x += xstride, ++w0, ++w1;
        if (++st == a.stages) st = 0, ph ^= 1;
      }
    }
    copies_landed();
  } else if (warp >= 14) {
    // ---- h from the first product's sums: units cta, cta + ctas, ...; a warp a
    // row, four hidden columns a lane.  The first round is a rehearsal on a spare
    // row: it brings the code into the instruction caches, which the weights
    // swept it from since the last call, while these warps are idle.
    for (int u = cta - ctas; u < A * G1; u += ctas) {
      const bool real = u >= 0;
      const int ei = real ? u / G1 : 0, g = real ? u - ei * G1 : 0;
      const Entry en = real ? ent[ei] : Entry{0, pairs, 2};
      if (real) wait_count(&unit_cnt[u], R1, abort, limit);
      __syncwarp();
#pragma unroll 1
      for (int n = warp - 14; n < en.n; n += 2) {
        float4 gate = make_float4(0.0f, 0.0f, 0.0f, 0.0f), up = gate;
        const float *src = a.sums + static_cast<int64_t>(real ? en.row + n : pairs) * 2 * a.I +
                           g * 128 + lane * 4;
#pragma unroll 4
        for (int c = 0; c < R1; ++c) {
          const float4 x = __ldcg(reinterpret_cast<const float4 *>(src));
          const float4 y = __ldcg(reinterpret_cast<const float4 *>(src + a.I));
          gate.x += x.x, gate.y += x.y, gate.z += x.z, gate.w += x.w;
          up.x += y.x, up.y += y.y, up.z += y.z, up.w += y.w;
          src += plane1;
        }
        hidden_row(a, gate, up, real ? en.row + n : pairs, g,
                   a.hs + ((real ? ei : a.max_entries) * G1 + g) * 32 + n);
      }
      fence_proxy_async_all();
      named_bar_sync(2, 64);
      if (real && warp == 14 && lane == 0) {
        __threadfence();
        atomicAdd(&ready[ei], 1u);
        atomicAdd(units_done, 1u);
      }
    }
  } else if (warp < 12) {
    // ---- epilogue: 256 threads, thread = (tile of the step, weight row)
    const int et = tid - 128, tile = et >> 7, row = et & 127, ew = et >> 5;
    const uint32_t tlane =
        tmem + ((static_cast<uint32_t>(warp & 3) * 32u) << 16) + tile * kCols;

    int st = 0, ph = 0;  // the next step's stage
    float acc[NT];
    int sg = 0, sph = 1;  // the next signal
    auto signal = [&] {
      __syncwarp();
      mbar_wait(&bars.sig_free[sg], sph, abort, limit);
      if (lane == 0) mbar_arrive(&bars.sig[sg]);
      if (++sg == kSignals) sg = 0, sph ^= 1;
    };
    // acc[i] = sum over `steps` K blocks of row i's partial sums from TMEM times
    // their scales.  pick: row i's TMEM column is lane i's xcol (a token), else i.
    auto sum_blocks = [&](int n, int steps, int xcol, bool pick, bool on) {
#pragma unroll
      for (int i = 0; i < NT; ++i) acc[i] = 0.0f;
#pragma unroll 1
      for (int i = 0; i < steps; ++i) {
        mbar_wait(&bars.tfull[st], ph, abort, limit);
        __syncwarp();
        tc_fence_after();
        const float *sc = scl + st * (NT + 4);
        uint32_t v[NT];
        float w[NT];
        if (on) {
          const uint32_t at = tlane + st * 2 * kCols;
          if (pick) {
#pragma unroll
            for (int c = 0; c < NT; ++c) {
              if (c >= n) break;
              tmem_ld1(at + __shfl_sync(0xFFFFFFFFu, xcol, c), v[c]);
            }
          } else {
            tmem_ld16(at, v);
            if (NT > 16 && n > 16) tmem_ld16(at + 16, v + (NT > 16 ? 16 : 0));
          }
          const float sw = sc[NT + tile];
#pragma unroll
          for (int c = 0; c < NT; c += 4) {
            if (c >= n) break;
            const float4 q = *reinterpret_cast<const float4 *>(sc + c);
            w[c] = q.x * sw, w[c + 1] = q.y * sw, w[c + 2] = q.z * sw, w[c + 3] = q.w * sw;
          }
          tmem_ld_wait();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.tempty[st]);
        if (++st == a.stages) st = 0, ph ^= 1;
        if (!on) continue;
#pragma unroll
        for (int c = 0; c < NT; ++c) {
          if (c >= n) break;
          acc[c] = fmaf(__uint_as_float(v[c]), w[c], acc[c]);
        }
      }
    };

    int qi = 0, qph = 0;
    // (the vote: a warp leaves whole, also when a wait ran out)
    while (__all_sync(0xFFFFFFFFu, mbar_wait(&bars.run_full[qi], qph, abort, limit))) {
      const Run run = bars.run[qi];
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.run_empty[qi]);
      if (++qi == kRunQueue) qi = 0, qph ^= 1;
      if (run.product == 0) break;
      const bool one = run.product == 1;
      const Entry en = ent[run.ei];
      sum_blocks(en.n, run.steps, one && lane < en.n ? tok[en.row + lane] : 0, one,
                 one || run.sub * 256 + tile * 128 < a.H);
      const int64_t pitch = one ? 2 * a.I : a.H;
      float *dst = one ? a.sums + run.plane * plane1 + tile * a.I + run.sub * 128 + row
                       : a.out + run.plane * plane2 + run.sub * 256 + et;
      dst += en.row * pitch;
      if (one || run.sub * 256 + et < a.H) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          if (n >= en.n) break;
          __stcg(dst, acc[n]);
          dst += pitch;
        }
      }
      if (one) signal();
    }
    signal();

    // ---- y when every run is done: 128 columns of a token a warp
    wait_count(all_done, ctas, abort, limit);
    __syncwarp();
    const int blocks = (a.H + 127) / 128;
    for (int i = ew * ctas + cta; i < a.M * blocks; i += ctas * kEpiWarps) {
      const int t = i / blocks, col = (i - t * blocks) * 128 + lane * 4;
      float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (col < a.H) {
#pragma unroll 1
        for (int k0 = 0; k0 < a.topk; k0 += 4) {  // four choices' loads in flight
          float4 o[4];
          int r[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            r[i] = row_of[t * kMoeMaxTopk + k0 + i];  // -1 from topk on
            o[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          }
#pragma unroll 2
          for (int c = 0; c < R2; ++c) {
            const float *src = a.out + c * plane2 + col;
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (r[i] >= 0) {
                const float4 q = __ldcg(
                    reinterpret_cast<const float4 *>(src + static_cast<int64_t>(r[i]) * a.H));
                o[i].x += q.x, o[i].y += q.y, o[i].z += q.z, o[i].w += q.w;
              }
          }
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (r[i] >= 0) {
              const float w = wrow[r[i]];
              v.x = fmaf(w, o[i].x, v.x), v.y = fmaf(w, o[i].y, v.y);
              v.z = fmaf(w, o[i].z, v.z), v.w = fmaf(w, o[i].w, v.w);
            }
        }
      }
      const uint32_t lo = bf16_bits(v.x) | (static_cast<uint32_t>(bf16_bits(v.y)) << 16);
      const uint32_t hi = bf16_bits(v.z) | (static_cast<uint32_t>(bf16_bits(v.w)) << 16);
      if (col < a.H)
        *reinterpret_cast<uint2 *>(a.y + static_cast<int64_t>(t) * a.H + col) = make_uint2(lo, hi);
    }
  }

  __syncthreads();
  if (tid == 0) {
    if (*abort) atomicMax(a.status, kStatusTimeout);
    bars.last = atom_add_acq_rel_gpu(leaving, 1) == static_cast<uint32_t>(ctas - 1);
  }
  if (warp == 1) tmem_dealloc(tmem, C::kTmemCols);
  __syncthreads();
  if (bars.last)  // the last CTA leaves the counters as it found them
    for (int i = tid; i < a.sync_words; i += kMoeThreads) a.sync[i] = 0;
}

int tokens_per_entry(int64_t M) { return M <= 16 ? 16 : 32; }

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

struct MoeLayout {
  size_t sync, xq, xs, hq, hs, sums, out, total;
  int max_entries, sync_words, planes;
};

// Counters of the largest call.  Their place and size are the same for all
// shapes, so that one workspace serves calls of several: they are zero between
// calls, and nothing else of any call lies there.
constexpr int kMoeSyncWords = 32 + (kMaxMoeExperts + kMoeMaxTokens * kMoeMaxTopk / 32) * (1 + 65536 / 128);

// Workspace: status word | counters | codes and scales of x (a row a
// token) and h (a row a token and expert) | the runs'
// sums of both products, a plane for each run of a sum, by hidden row
MoeLayout moe_layout(int64_t M, int64_t E, int64_t H, int64_t I, int64_t topk) {
  MoeLayout l;
  const int64_t P = M * topk, NT = tokens_per_entry(M);
  const int64_t KB1 = (H + 127) / 128, G1 = I / 128;
  l.max_entries = static_cast<int>((E < P ? E : P) + P / NT);
  l.sync_words = static_cast<int>(32 + l.max_entries * (1 + G1));
  size_t at = 256;
  auto take = [&](int64_t bytes) {
    const size_t here = at;
    at += up256(static_cast<size_t>(bytes));
    return here;
  };
  l.sync = take(kMoeSyncWords * 4);
  l.xq = take(M * KB1 * 128);
  l.xs = take(M * KB1 * 4);
  l.hq = take((P + 1) * I);  // and a spare row
  l.hs = take((l.max_entries + 1) * G1 * 32 * 4);
  l.planes = M <= 16 ? 8 : 4;  // most runs of a sum
  auto planes = [&](int64_t KB) { return KB < l.planes ? KB : l.planes; };
  l.sums = take(planes(KB1) * (P + 1) * 2 * I * 4);
  l.out = take(planes(G1) * P * H * 4);
  l.total = at;
  return l;
}

}  // namespace

size_t moe_workspace(int64_t M, int64_t E, int64_t H, int64_t I, int64_t topk) {
  return moe_layout(M, E, H, I, topk).total;
}

cudaError_t launch_moe_layer(MoeArgs a, const void *w13, const void *w2, void *ws,
                             const DeviceInfo &dev, cudaStream_t st) {
  const int ctas = dev.num_sms < kMoeMaxCtas ? dev.num_sms : kMoeMaxCtas;
  const MoeLayout l = moe_layout(a.M, a.E, a.H, a.I, a.topk);
  uint8_t *base = static_cast<uint8_t *>(ws);
  a.status = reinterpret_cast<uint32_t *>(base);
  a.sync = reinterpret_cast<uint32_t *>(base + l.sync);
  a.xq = base + l.xq;
  a.xs = reinterpret_cast<float *>(base + l.xs);
  a.hq = base + l.hq;
  a.hs = reinterpret_cast<float *>(base + l.hs);
  a.sums = reinterpret_cast<float *>(base + l.sums);
  a.out = reinterpret_cast<float *>(base + l.out);
  a.planes = l.planes;
  a.max_entries = l.max_entries;
  a.sync_words = l.sync_words;
  const int64_t P = static_cast<int64_t>(a.M) * a.topk, KB1 = (a.H + 127) / 128;
  const int NT = tokens_per_entry(a.M);
  const size_t fixed = 1024 + static_cast<size_t>(a.M) * kMoeMaxTopk * 8 + P * 6 +
                       static_cast<size_t>(l.max_entries) * sizeof(Entry) +
                       static_cast<size_t>(a.E) * 12;
  const size_t stage = (NT == 16 ? MoeCfg<16>::kStage : MoeCfg<32>::kStage) + (NT + 4) * 4;
  const size_t room = dev.max_smem_optin - 1024;  // the static part
  a.stages = static_cast<int>((room - fixed) / stage);
  const int most = NT == 16 ? MoeCfg<16>::kMaxStages : MoeCfg<32>::kMaxStages;
  if (a.stages > most) a.stages = most;

  const size_t smem = fixed + a.stages * stage;

  CUtensorMap m13, m2, mx, mh;
  if (!make_kmajor_map(&m13, w13, static_cast<int64_t>(a.E) * 2 * a.I, a.H, 128) ||
      !make_kmajor_map(&m2, w2, static_cast<int64_t>(a.E) * a.H, a.I, 128) ||
      !make_kmajor_map(&mx, a.xq, a.M, KB1 * 128, 16) || !make_kmajor_map(&mh, a.hq, P + 1, a.I, 16))
    return cudaErrorInvalidValue;
  auto run = [&](auto nt) {
    constexpr auto kern = moe_layer_kernel<decltype(nt)::value>;
    cudaError_t e = allow_smem<moe_layer_kernel<decltype(nt)::value>>(
        static_cast<int>(dev.max_smem_optin) - 1024);
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
  return NT == 16 ? run(std::integral_constant<int, 16>{}) : run(std::integral_constant<int, 32>{});
}

}  // namespace fp8bq
