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
// output rows), and the steps into runs that a CTA takes whole: one long run
// each, and short ones that whoever is done first takes (dealt equally in
// advance, the slowest SMs finished up to a third later than the rest: 276
// against 240 us for 16 tokens of 32 experts of 7168 x 2048).  The epilogue
// warps leave each sum, or their part of one that a run's end cuts, in the
// workspace and go on; they wait for nobody but the tensor core.  Two warps of
// a CTA that the unit names join the parts of the first product, in run order,
// and make h of them; the parts of the second are joined when all is done, each
// CTA taking its share of the outputs.  The runs' bounds and every order of
// addition follow from the sizes and the routing alone, so results repeat bit
// for bit whoever took which run.
//
// The tensor core sees the weights as the 128 rows of A and up to NT tokens as
// the columns of B (tcgen05.mma, M = 128).  In the first product the columns
// are all tokens, whoever chose the expert: x then needs no order by expert
// and is quantised while the routing is still going on, and the epilogue reads
// the chosen tokens' columns alone.  In the second they are the entry's hidden
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

// Warps: 0 weight copies, 2 activation copies, 1, 3 and 12 MMA issuers, 4 to 11
// the epilogue, 13 idle, 14 and 15 finish h.  One MMA instruction of so few
// columns takes its issuer about 0.06 us: a single issuer set the pace (0.75 us
// for a step's eight, HBM half idle), so three take the stages in turn.
constexpr int kMoeThreads = 512;
constexpr int kIssuers = 3;
constexpr int kEpi = 256;
constexpr int kEpiWarps = 8;
constexpr int kTileBytes = 128 * 128;
constexpr int kMaxRing = 8;
constexpr int kRunQueue = 4;
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

// How `steps` steps are cut into runs.  Run c < parts is CTA c's own; together
// they hold `fixed` steps, all of them where a CTA's share is small, else three
// fifths.  The runs after them, of q steps, are taken in turn.
struct Deal {
  uint32_t steps, parts, fixed, q, runs;
  __device__ __forceinline__ Deal(int steps_, int ctas, int q_min) {
    steps = steps_, parts = min(steps_, ctas);
    const bool small = steps_ < 12 * ctas;
    fixed = small ? steps : steps / 5 * 3;
    q = max(q_min, (steps_ + 12 * ctas - 1) / (12 * ctas));
    runs = parts + (steps - fixed + q - 1) / q;
  }
  // Products below stay below 2^32: no GPU's memory holds 2^24 steps' weights.
  __device__ __forceinline__ int begin(uint32_t c) const {  // also the end of run c - 1
    if (c >= runs) return steps;
    return c <= parts ? (parts ? c * fixed / parts : 0)
                      : fixed + (c - parts) * q;
  }
  __device__ __forceinline__ int owner(uint32_t s) const {  // the run that has step s
    return s < fixed ? ((s + 1) * parts - 1) / fixed : parts + (s - fixed) / q;
  }
};
constexpr int kMaxRuns = 960;  // 160 + 0.4 * 12 * 160, rounded up

// What the weight warp hands to the others: a run of one of the products.
struct Run {
  int product;  // 1, 2; 0: no more
  int id, begin, end;
};

struct MoeBars {
  uint64_t full_w[kMaxRing], full_b[kMaxRing], empty[kMaxRing];
  uint64_t tfull[kMaxRing], tempty[kMaxRing];
  uint64_t run_full[kRunQueue], run_empty[kRunQueue];
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
        const float v = value_of(best);
        const uint32_t near = key_of(v - (1e-6f + 4e-7f * fabsf(v)));
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
    float v = 0.0f;
    if (got_at >= 0) {
      const float x = a.bias ? fminf(__ldg(row + got_at), 3.402823466e38f) : value_of(got);
      v = a.score == 0 ? expf(x - value_of(top)) / denom : sigmoid(x);
    }
    if (a.renorm) {
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

// A part of a cut sum, [rows][256]: a run is cut at most in its first unit (slot
// 0) and in its last.
__device__ __forceinline__ int64_t part_at(int run, int slot, int rows) {
  return (static_cast<int64_t>(run) * 2 + slot) * rows * 256;
}
// The runs that hold unit u's sum, and the slot of the first one's part (the
// others begin inside the unit: slot 0).
struct Parts {
  int c0, c1, slot0;
  __device__ __forceinline__ Parts(const Deal &d, int u, int KB)
      : c0(d.owner(u * KB)), c1(d.owner(u * KB + KB - 1)), slot0(d.begin(c0) / KB == u ? 0 : 1) {}
};

// One hidden row's 128 columns of group g by a warp: h = silu(gate) * up, codes
// and scale.
__device__ void hidden_row(const MoeArgs &a, float4 gate, float4 up, int row, int g, int pairs) {
  const int lane = threadIdx.x & 31;
  const float f[4] = {gate.x * sigmoid(gate.x) * up.x, gate.y * sigmoid(gate.y) * up.y,
                      gate.z * sigmoid(gate.z) * up.z, gate.w * sigmoid(gate.w) * up.w};
  float sc;
  const uint32_t code = quant4(f, &sc);
  *reinterpret_cast<uint32_t *>(a.hq + static_cast<int64_t>(row) * a.I + g * 128 + lane * 4) = code;
  if (lane == 0) a.hs[g * (pairs + 1) + row] = sc;
}

template <int NT>
struct MoeCfg {
  static constexpr int kTokens = NT == 16 ? 16 : kMoeMaxTokens;
  static constexpr int kStage = 2 * kTileBytes + kTokens * 128;
  static constexpr int kCols = kTokens;              // TMEM columns of one partial tile
  static constexpr int kMaxStages = NT == 16 ? 8 : 4;  // a stage has a TMEM buffer of two tiles
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
  const int J = (a.H + 255) / 256, rows = min(a.M, NT);

  uint8_t *ring = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  float *wgt = reinterpret_cast<float *>(ring + a.stages * kStage);  // [M][16]: weight by choice
  float *wrow = wgt + a.M * kMoeMaxTopk;                    // [pairs]: by hidden row
  Entry *ent = reinterpret_cast<Entry *>(wrow + pairs);     // [max_entries]
  uint32_t *mask = reinterpret_cast<uint32_t *>(ent + a.max_entries);  // [E][2]: tokens' bits
  int *first = reinterpret_cast<int *>(mask + 2 * a.E);     // [E]: first hidden row
  short *ids = reinterpret_cast<short *>(first + a.E);      // [M][16], -1: none
  short *row_of = ids + a.M * kMoeMaxTopk;                  // [M][16]: hidden row, -1: none
  short *tok = row_of + a.M * kMoeMaxTopk;                  // [pairs]: token of a hidden row
  short *ent_of = tok + pairs;                              // [pairs]: its entry

  uint32_t *const all_quant = a.sync;       // CTAs whose share of x is quantised
  uint32_t *const all_done = a.sync + 1;    // epilogue warps without a run left
  uint32_t *const leaving = a.sync + 2;
  uint32_t *const claim1 = a.sync + 3;      // short runs taken
  uint32_t *const claim2 = a.sync + 4;
  uint32_t *const units_done = a.sync + 5;  // hidden groups published,
  uint32_t *const ready = a.sync + 32;      // [entries]: by entry
  uint32_t *const unit_cnt = ready + a.max_entries;  // [entries * G1]: sums left, by epilogue warp
  const uint32_t quant_ctas = min(ctas, a.M * KB1);

  if (tid == 0) {
    for (int i = 0; i < a.stages; ++i) {
      mbar_init(&bars.full_w[i], 1);
      mbar_init(&bars.full_b[i], 1);
      mbar_init(&bars.empty[i], 1);
    }
    for (int i = 0; i < a.stages; ++i) {
      mbar_init(&bars.tfull[i], 1);
      mbar_init(&bars.tempty[i], kEpiWarps);
    }
    for (int i = 0; i < kRunQueue; ++i) {
      mbar_init(&bars.run_full[i], 1);
      mbar_init(&bars.run_empty[i], 1 + kIssuers + kEpiWarps);
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
    tmem_alloc(&bars.tmem, 512);
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
      for (int k = 0; k < n; k += NT, ++ee) {
        ent[ee] = Entry{e, rr + k, min(NT, n - k)};
        for (int r = k; r < min(n, k + NT); ++r) ent_of[rr + r] = static_cast<short>(ee);
      }
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
  const Deal d1(A * G1 * KB1, ctas, 6), d2(J * A * KB2, ctas, 4);
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
      for (uint32_t c = cta; c < d1.runs && ok;) {
        const int b = d1.begin(c), e = d1.begin(c + 1);
        hand(Run{1, static_cast<int>(c), b, e});
        int u = b / KB1, kb = b - u * KB1, ei = u / G1, g = u - ei * G1;
        for (int left = e - b; left > 0 && ok;) {
          const int r = ent[ei].e * 2 * a.I + g * 128;
          const float *sc = a.s13 + (static_cast<int64_t>(ent[ei].e) * 2 * G1 + g) * KB1 + kb;
          prefetch_l2(sc);
          prefetch_l2(sc + G1 * KB1);
          for (; kb < KB1 && left > 0 && ok; ++kb, --left) stage(&map13, kb, r, r + a.I, true);
          kb = 0;
          if (++g == G1) g = 0, ++ei;
        }
        c = d1.runs > d1.parts ? d1.parts + atomicAdd(claim1, 1u) : d1.runs;
      }
      for (uint32_t c = cta; c < d2.runs && ok;) {
        const int b = d2.begin(c), e = d2.begin(c + 1);
        hand(Run{2, static_cast<int>(c), b, e});
        int u = b / KB2, kb = b - u * KB2, j = u / A, ei = u - j * A;
        for (int left = e - b; left > 0 && ok;) {
          const int r = ent[ei].e * a.H + j * 256;
          const bool two = j * 256 + 128 < a.H;
          prefetch_l2(a.s2 + (static_cast<int64_t>(ent[ei].e) * ((a.H + 127) / 128) + 2 * j) * KB2);
          for (; kb < KB2 && left > 0 && ok; ++kb, --left) stage(&map2, kb, r, r + 128, two);
          kb = 0;
          if (++ei == A) ei = 0, ++j;
        }
        c = d2.runs > d2.parts ? d2.parts + atomicAdd(claim2, 1u) : d2.runs;
      }
      if (ok) hand(Run{0, 0, 0, 0});
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
        const CUtensorMap *map = run.product == 1 ? &mapx : &maph;
        const int KB = run.product == 1 ? KB1 : KB2;
        if (run.product == 1 && !quantised) {
          ok = quantised = wait_count(all_quant, quant_ctas, abort, limit);
          fence_proxy_async_all();
        }
        int u = run.begin / KB, kb = run.begin - u * KB, ei = u % A;
        for (int left = run.end - run.begin; left > 0 && ok;) {
          int row = 0, boxes = xboxes;
          if (run.product == 2) {
            if (!hidden) {
              hidden = ld_acquire_gpu(units_done) >= static_cast<uint32_t>(A * G1);
              if (!hidden) ok = wait_count(&ready[ei], G1, abort, limit);
              fence_proxy_async_all();
            }
            row = ent[ei].row, boxes = (ent[ei].n + 15) / 16;
          }
          for (; kb < KB && left > 0 && ok; ++kb, --left) {
            ok = mbar_wait(&bars.empty[st], ph, abort, limit);
            if (!ok) break;
            uint8_t *dst = ring + st * kStage + 2 * kTileBytes;
            mbar_arrive_expect_tx(&bars.full_b[st], boxes * 2048);
            for (int i = 0; i < boxes; ++i)
              tma_load_2d(dst + i * 2048, map, &bars.full_b[st], kb * 128, row + i * 16);
            ++it;
            if (++st == a.stages) st = 0, ph ^= 1;
          }
          kb = 0;
          if (++ei == A) ei = 0;
        }
      }
      if (!ok)
        for (int i = max(0, it - a.stages); i < it; ++i)
          mbar_wait(&bars.full_b[i % a.stages], (i / a.stages) & 1, never, limit);
    }
    __syncwarp();
  } else if (warp == 1 || warp == 3 || warp == 12) {
    if (lane == 0) {  // ---- MMAs
      // A stage, and the TMEM buffer of the same number, belong to one issuer:
      // a parity wait tells two phases apart, not three, so whoever waits for
      // a stage's phase must have seen the one before.
      const int st0 = warp < 4 ? warp >> 1 : warp - 10;
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
        const int it1 = it0 + run.end - run.begin;
        while (it < it1 && st0 < a.stages) {
          int n = a.M;
          bool two = true;
          if (run.product == 2) {
            const int u = (run.begin + it - it0) / KB2, j = u / A;
            n = ent[u - j * A].n;
            two = j * 256 + 128 < a.H;
          }
          ok = mbar_wait(&bars.tempty[st], ph ^ 1, abort, limit) &&
               mbar_wait(&bars.full_w[st], ph, abort, limit) &&
               mbar_wait(&bars.full_b[st], ph, abort, limit);
          if (!ok) break;
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
  } else if (warp >= 14) {
    // ---- h from the first product's sums: units cta, cta + ctas, ...; a warp a
    // row, four hidden columns a lane.  The first round is a rehearsal on a spare
    // row: it brings the code into the instruction caches, which the weights
    // swept it from since the last call, while these warps are idle.
    for (int u = cta - ctas; u < A * G1; u += ctas) {
      const bool real = u >= 0;
      const Parts p(d1, real ? u : 0, KB1);
      const int ei = real ? u / G1 : 0, g = real ? u - ei * G1 : 0;
      const Entry en = real ? ent[ei] : Entry{0, pairs, 2};
      if (real) wait_count(&unit_cnt[u], (p.c1 - p.c0 + 1) * kEpiWarps, abort, limit);
      __syncwarp();
#pragma unroll 1
      for (int n = warp - 14; n < en.n; n += 2) {
        float4 gate = make_float4(0.0f, 0.0f, 0.0f, 0.0f), up = gate;
#pragma unroll 4
        for (int c = p.c0; c <= p.c1; ++c) {
          const float *src = a.part1 + part_at(c, c == p.c0 ? p.slot0 : 0, rows) + n * 256;
          int far = 128;
          if (p.c0 == p.c1)  // whole
            src = a.sums + static_cast<int64_t>(en.row + (real ? n : 0)) * 2 * a.I + g * 128, far = a.I;
          const float4 x = __ldcg(reinterpret_cast<const float4 *>(src + lane * 4));
          const float4 y = __ldcg(reinterpret_cast<const float4 *>(src + far + lane * 4));
          gate.x += x.x, gate.y += x.y, gate.z += x.z, gate.w += x.w;
          up.x += y.x, up.y += y.y, up.z += y.z, up.w += y.w;
        }
        hidden_row(a, gate, up, real ? en.row + n : pairs, g, pairs);
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

    int slot = 0, phase = 0;  // the next step's TMEM buffer
    float acc[NT];
    // acc[i] = sum over K blocks [kb0, kb1) of a unit: partial sums from TMEM
    // times the weight block's scale (wscale[kb]) and row i's (xscale[kb *
    // xstride + xrow], xrow held by lane i).  pick: row i's TMEM column is
    // lane i's xrow (a token), else i.
    auto sum_blocks = [&](int n, int kb0, int kb1, const float *wscale, const float *xscale,
                          int xstride, int xrow, bool pick, bool on) {
#pragma unroll
      for (int i = 0; i < NT; ++i) acc[i] = 0.0f;
      auto xs_at = [&](int kb) {
        return kb < kb1 && lane < n ? __ldcg(xscale + kb * xstride + xrow) : 0.0f;
      };
      // scales three blocks ahead
      float x0 = xs_at(kb0), x1 = xs_at(kb0 + 1), x2 = xs_at(kb0 + 2), sw = 0.0f;
#pragma unroll 1
      for (int kb = kb0; kb < kb1; ++kb) {
        const float sx = x0;
        x0 = x1, x1 = x2, x2 = xs_at(kb + 3);
        if (((kb - kb0) & 31) == 0)
          sw = on && kb + lane < kb1 ? __ldg(wscale + kb + lane) : 0.0f;
        const int sl = slot;
        mbar_wait(&bars.tfull[sl], phase, abort, limit);
        __syncwarp();
        if (++slot == a.stages) slot = 0, phase ^= 1;
        tc_fence_after();
        uint32_t v[NT];
        if (on) {
          const uint32_t at = tlane + sl * 2 * kCols;
          if (pick) {
#pragma unroll
            for (int c = 0; c < NT; ++c) {
              if (c >= n) break;
              tmem_ld1(at + __shfl_sync(0xFFFFFFFFu, xrow, c), v[c]);
            }
          } else {
            tmem_ld16(at, v);
            if (NT > 16 && n > 16) tmem_ld16(at + 16, v + (NT > 16 ? 16 : 0));
          }
          tmem_ld_wait();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.tempty[sl]);
        if (!on) continue;
        const float w = sx * __shfl_sync(0xFFFFFFFFu, sw, (kb - kb0) & 31);
#pragma unroll
        for (int c = 0; c < NT; ++c) {
          if (c >= n) break;
          acc[c] = fmaf(__uint_as_float(v[c]), __shfl_sync(0xFFFFFFFFu, w, c), acc[c]);
        }
      }
    };

    bool quantised = false, hidden = false;
    int qi = 0, qph = 0;
    // (the vote: a warp leaves whole, also when a wait ran out)
    while (__all_sync(0xFFFFFFFFu, mbar_wait(&bars.run_full[qi], qph, abort, limit))) {
      const Run run = bars.run[qi];
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.run_empty[qi]);
      if (++qi == kRunQueue) qi = 0, qph ^= 1;
      if (run.product == 0) break;

      if (run.product == 1) {
        if (!quantised) {
          wait_count(all_quant, quant_ctas, abort, limit);
          __syncwarp();
          quantised = true;
        }
        for (int s = run.begin; s < run.end;) {
          const int u = s / KB1, kb0 = s - u * KB1, kb1 = min(KB1, kb0 + run.end - s);
          const int ei = u / G1, g = u - ei * G1;
          const Entry en = ent[ei];
          sum_blocks(en.n, kb0, kb1,
                     a.s13 + (static_cast<int64_t>(en.e) * 2 * G1 + tile * G1 + g) * KB1, a.xs,
                     a.M, lane < en.n ? tok[en.row + lane] : 0, true, true);
          float *dst;
          int pitch;
          if (kb1 - kb0 == KB1) {
            dst = a.sums + static_cast<int64_t>(en.row) * 2 * a.I + tile * a.I + g * 128 + row;
            pitch = 2 * a.I;
          } else {
            dst = a.part1 + part_at(run.id, run.begin / KB1 == u ? 0 : 1, rows) + et, pitch = 256;
          }
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            if (n >= en.n) break;
            __stcg(dst + static_cast<int64_t>(n) * pitch, acc[n]);
          }
          __syncwarp();
          if (lane == 0) red_release_gpu(&unit_cnt[u], 1);
          s += kb1 - kb0;
        }
        continue;
      }

      for (int s = run.begin; s < run.end;) {
        const int u = s / KB2, kb0 = s - u * KB2, kb1 = min(KB2, kb0 + run.end - s);
        const int j = u / A, ei = u - j * A, col = j * 256 + et;
        const Entry en = ent[ei];
        const bool on = j * 256 + tile * 128 < a.H;
        if (!hidden) {
          hidden = __all_sync(0xFFFFFFFFu,
                              ld_acquire_gpu(units_done) >= static_cast<uint32_t>(A * G1));
          if (!hidden) wait_count(&ready[ei], G1, abort, limit);
          __syncwarp();
        }
        sum_blocks(en.n, kb0, kb1,
                   a.s2 + (static_cast<int64_t>(en.e) * ((a.H + 127) / 128) + 2 * j + tile) * KB2,
                   a.hs, pairs + 1, en.row + lane, false, on);
        // a whole sum is a row of `out`; a cut one a part of its run
        float *dst;
        int pitch;
        if (kb1 - kb0 == KB2) {
          dst = a.out + static_cast<int64_t>(en.row) * a.H + col, pitch = a.H;
        } else {
          dst = a.part2 + part_at(run.id, run.begin / KB2 == u ? 0 : 1, rows) + et, pitch = 256;
        }
        if (col < a.H) {
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            if (n >= en.n) break;
            __stcg(dst + static_cast<int64_t>(n) * pitch, acc[n]);
          }
        }
        s += kb1 - kb0;
      }
    }

    // ---- y when every run is done: 128 columns of a token a warp
    __syncwarp();
    if (lane == 0) red_release_gpu(all_done, 1);
    wait_count(all_done, ctas * kEpiWarps, abort, limit);
    __syncwarp();
    const int blocks = (a.H + 127) / 128;
    for (int i = ew * ctas + cta; i < a.M * blocks; i += ctas * kEpiWarps) {
      const int t = i / blocks, blk = i - t * blocks, j = blk / 2, col = blk * 128 + lane * 4;
      // lane k finds the parts of choice k
      const int rk = lane < kMoeMaxTopk ? row_of[t * kMoeMaxTopk + lane] : -1;
      const int ek = rk >= 0 ? ent_of[rk] : 0;
      const Parts pk(d2, j * A + ek, KB2);
      const int nk = rk >= 0 ? rk - ent[ek].row : 0;
      const float wk = rk >= 0 ? wrow[rk] : 0.0f;
      float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
      for (int k = 0; k < a.topk; ++k) {
        const int r = __shfl_sync(0xFFFFFFFFu, rk, k), n = __shfl_sync(0xFFFFFFFFu, nk, k);
        const int c0 = __shfl_sync(0xFFFFFFFFu, pk.c0, k), c1 = __shfl_sync(0xFFFFFFFFu, pk.c1, k);
        const int slot0 = __shfl_sync(0xFFFFFFFFu, pk.slot0, k);
        const float w = __shfl_sync(0xFFFFFFFFu, wk, k);
        if (r < 0 || col >= a.H) continue;
        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int c = c0; c <= c1; ++c) {
          const float *src = c0 == c1 ? a.out + static_cast<int64_t>(r) * a.H + col
                                      : a.part2 + part_at(c, c == c0 ? slot0 : 0, rows) + n * 256 +
                                            (blk & 1) * 128 + lane * 4;
          const float4 q = __ldcg(reinterpret_cast<const float4 *>(src));
          o.x += q.x, o.y += q.y, o.z += q.z, o.w += q.w;
        }
        v.x = fmaf(w, o.x, v.x), v.y = fmaf(w, o.y, v.y);
        v.z = fmaf(w, o.z, v.z), v.w = fmaf(w, o.w, v.w);
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
  if (warp == 1) tmem_dealloc(tmem, 512);
  __syncthreads();
  if (bars.last)  // the last CTA leaves the counters as it found them
    for (int i = tid; i < a.sync_words; i += kMoeThreads) a.sync[i] = 0;
}

int tokens_per_entry(int64_t M) { return M <= 16 ? 16 : 32; }

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

struct MoeLayout {
  size_t sync, xq, xs, hq, hs, sums, out, part1, part2, total;
  int max_entries;
  int sync_words;
};

// Workspace: status word | counters | codes and scales of x (a row a
// token) and h (a row a token and expert) | the sums of
// both products by hidden row | parts of cut sums of both products, two for each run
MoeLayout moe_layout(int64_t M, int64_t E, int64_t H, int64_t I, int64_t topk) {
  MoeLayout l;
  const int64_t P = M * topk, NT = tokens_per_entry(M);
  const int64_t KB1 = (H + 127) / 128, G1 = I / 128, rows = M < NT ? M : NT;
  l.max_entries = static_cast<int>((E < P ? E : P) + P / NT);
  l.sync_words = static_cast<int>(32 + l.max_entries * (1 + G1));
  size_t at = 256;
  auto take = [&](int64_t bytes) {
    const size_t here = at;
    at += up256(static_cast<size_t>(bytes));
    return here;
  };
  l.sync = take(l.sync_words * 4);
  l.xq = take(M * KB1 * 128);
  l.xs = take(M * KB1 * 4);
  l.hq = take((P + 1) * I);  // and a spare row
  l.hs = take((P + 1) * G1 * 4);
  l.sums = take((P + 1) * 2 * I * 4);
  l.out = take(P * H * 4);
  l.part1 = take(static_cast<int64_t>(kMaxRuns) * 2 * rows * 256 * 4);
  l.part2 = take(static_cast<int64_t>(kMaxRuns) * 2 * rows * 256 * 4);
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
  a.part1 = reinterpret_cast<float *>(base + l.part1);
  a.part2 = reinterpret_cast<float *>(base + l.part2);
  a.max_entries = l.max_entries;
  a.sync_words = l.sync_words;
  const int64_t P = static_cast<int64_t>(a.M) * a.topk, KB1 = (a.H + 127) / 128;
  const int NT = tokens_per_entry(a.M);
  const size_t fixed = 1024 + static_cast<size_t>(a.M) * kMoeMaxTopk * 8 + P * 8 +
                       static_cast<size_t>(l.max_entries) * sizeof(Entry) +
                       static_cast<size_t>(a.E) * 12;
  const size_t stage = NT == 16 ? MoeCfg<16>::kStage : MoeCfg<32>::kStage;
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
