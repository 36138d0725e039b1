// rope.cu -- RMSNorm of every query and key head and the rotary embedding in
// one pass over the QKV projection's output.
//
// Per head v of D values (FP32 throughout, one rounding to BF16 at the end):
//   n = v * rsqrt(mean(v^2) + eps) * gamma             (gamma given; else n = v)
//   pairs (a, b) of the first `rot` values:  a' = a cos - b sin, b' = b cos + a sin
// with cos, sin from the row of the FP32 table that the token's position names;
// pairs are (i, i + rot/2), or (2i, 2i+1) in the interleaved form.
//
// Bound by HBM: every q and k value is read once and written once (4 bytes a
// value).  A head belongs to G lanes of a warp, 16 values a lane: in the split
// form a lane holds 8 values of the first half and their 8 partners of the
// second, so a rotation needs no exchange and every access is 16 bytes.  The
// table row and the gains stay in registers over the heads that a warp walks.
#include "common.cuh"
#include "ptx.cuh"
#include "quant_math.cuh"

namespace fp8bq {
namespace {

// One warp a CTA, 28 of them an SM (72 registers): 51 us for 8192 tokens of 72
// heads of 128, against 57 with four warps a CTA, whose last rounds leave SMs idle
// longer; without the loads of the next step 66.
constexpr int kRopeThreads = 32;
constexpr int kRopeBlocks = 28;

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// 8 table entries (32-byte aligned)
__device__ __forceinline__ void load8(const float *p, float (&f)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4 *>(p));
  const float4 b = __ldg(reinterpret_cast<const float4 *>(p) + 1);
  f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
  f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
}

template <int G>  // lanes a head (16 values each): 4, 8, 16 or 32
__global__ void __launch_bounds__(kRopeThreads, kRopeBlocks) qk_norm_rope_kernel(const RopeArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const int64_t warp = static_cast<int64_t>(blockIdx.x) * (kRopeThreads / 32) + (threadIdx.x >> 5);
  const int64_t t = warp / a.chunks;
  if (t >= a.T) return;
  const int h0 = static_cast<int>(warp % a.chunks) * a.chunk_heads;
  const int heads = a.HQ + a.HK;
  const int h1 = min(heads, h0 + a.chunk_heads);
  const int j = lane % G;
  const bool on = j * 16 < a.D;  // lanes past the head's end only take part in the sums
  const bool turn = j * 16 < a.rot;
  // element offsets of this lane's two 8-value words within a head
  const int lo = a.interleaved || !turn ? j * 16 : j * 8;
  const int hi = a.interleaved || !turn ? lo + 8 : lo + a.rot / 2;

  const int64_t pos = a.pos_is64 ? static_cast<const int64_t *>(a.pos)[t]
                                 : static_cast<const int32_t *>(a.pos)[t];
  const bool known = pos >= 0 && pos < a.P;  // other tokens are padding: zeros
  float cs[8], sn[8];
  if (turn && known) {
    const float *row = a.table + pos * a.rot + j * 8;
    load8(row, cs);
    load8(row + a.rot / 2, sn);
  }
  // gains as packed BF16 words, queries' and keys'
  uint4 gq[2] = {}, gk[2] = {};
  if (on && a.gq) {
    gq[0] = __ldg(reinterpret_cast<const uint4 *>(a.gq + lo));
    gq[1] = __ldg(reinterpret_cast<const uint4 *>(a.gq + hi));
  }
  if (on && a.gk) {
    gk[0] = __ldg(reinterpret_cast<const uint4 *>(a.gk + lo));
    gk[1] = __ldg(reinterpret_cast<const uint4 *>(a.gk + hi));
  }
  const float inv_d = 1.0f / static_cast<float>(a.D);

  // the next step's heads are loaded while this one's are computed
  const uint16_t *const qs = a.q + t * a.q_ts, *const ks = a.k + t * a.k_ts;
  auto load = [&](int h, uint4 (&v)[2]) {
    if (h >= h1 || !on) return;
    const uint16_t *src = h < a.HQ ? qs + h * a.q_hs : ks + (h - a.HQ) * a.k_hs;
    v[0] = *reinterpret_cast<const uint4 *>(src + lo);
    v[1] = *reinterpret_cast<const uint4 *>(src + hi);
  };
  uint4 ahead[2] = {};
  load(h0 + lane / G, ahead);
#pragma unroll 1
  for (int hb = h0; hb < h1; hb += 32 / G) {
    const int h = hb + lane / G;
    const bool live = h < h1 && on;
    const bool isq = h < a.HQ;
    const int hh = isq ? h : h - a.HQ;
    uint16_t *dst = isq ? a.qo + t * a.qo_ts + hh * a.qo_hs : a.ko + t * a.ko_ts + hh * a.ko_hs;
    const uint4 v[2] = {ahead[0], ahead[1]};
    load(h + 32 / G, ahead);
    float f[16];
    unpack16(v, f);
    if (isq ? a.gq != nullptr : a.gk != nullptr) {
      float ss = 0.0f;
#pragma unroll
      for (int i = 0; i < 16; ++i) ss = fmaf(f[i], f[i], ss);
      // every lane of the warp has the same trip count, and the lanes of one
      // head take the same branch
      const uint32_t mask = G == 32 ? 0xFFFFFFFFu : ((1u << G) - 1u) << (lane / G * G);
#pragma unroll
      for (int d = G / 2; d > 0; d >>= 1) ss += __shfl_xor_sync(mask, ss, d);
      const float r = rsqrtf(fmaf(ss, inv_d, a.eps));
      const uint4 gp[2] = {isq ? gq[0] : gk[0], isq ? gq[1] : gk[1]};
      float g[16];
      unpack16(gp, g);
#pragma unroll
      for (int i = 0; i < 16; ++i) f[i] = f[i] * r * g[i];
    }
    if (!live) continue;
    if (turn && known) {
      if (a.interleaved) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float x = f[2 * i], y = f[2 * i + 1];
          f[2 * i] = x * cs[i] - y * sn[i];
          f[2 * i + 1] = y * cs[i] + x * sn[i];
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float x = f[i], y = f[8 + i];
          f[i] = x * cs[i] - y * sn[i];
          f[8 + i] = y * cs[i] + x * sn[i];
        }
      }
    }
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = known ? pack_bf16(f[2 * i], f[2 * i + 1]) : 0u;
    *reinterpret_cast<uint4 *>(dst + lo) = make_uint4(w[0], w[1], w[2], w[3]);
    *reinterpret_cast<uint4 *>(dst + hi) = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

}  // namespace

cudaError_t launch_qk_norm_rope(RopeArgs a, int num_sms, cudaStream_t st) {
  const int G = a.D <= 64 ? 4 : a.D <= 128 ? 8 : a.D <= 256 ? 16 : 32;
  const int per = 32 / G;  // heads a warp takes at once
  const int heads = a.HQ + a.HK;
  // A warp walks as many heads of its token as leave 32 warps to every SM, so
  // that the table row and the gains are read once for them; with few tokens
  // each warp takes one step and the latency of one is all there is.
  const int64_t steps = (heads + per - 1) / per;
  const int64_t want = static_cast<int64_t>(num_sms) * 32;
  int64_t chunks = (want + a.T - 1) / a.T;
  if (chunks > steps) chunks = steps;
  const int64_t steps_each = (steps + chunks - 1) / chunks;
  a.chunk_heads = static_cast<int>(steps_each * per);
  a.chunks = static_cast<int>((steps + steps_each - 1) / steps_each);
  const int64_t warps = a.T * a.chunks;
  const int64_t blocks = (warps + kRopeThreads / 32 - 1) / (kRopeThreads / 32);
  const dim3 grid(static_cast<unsigned>(blocks)), block(kRopeThreads);
  switch (G) {
    case 4: return launch_pdl(qk_norm_rope_kernel<4>, grid, block, 0, st, a);
    case 8: return launch_pdl(qk_norm_rope_kernel<8>, grid, block, 0, st, a);
    case 16: return launch_pdl(qk_norm_rope_kernel<16>, grid, block, 0, st, a);
    default: return launch_pdl(qk_norm_rope_kernel<32>, grid, block, 0, st, a);
  }
}

}  // namespace fp8bq
