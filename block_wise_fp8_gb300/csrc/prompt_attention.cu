// prompt_attention.cu -- causal attention over whole prompts: packed sequences of
// different lengths, grouped heads.
//
// Per sequence (rows offsets[s] .. offsets[s+1]-1), token i and head h:
//   s_j = scale * q_i . k_j for j <= i,  y_i = sum_j softmax(s)_j v_j
// with the maximum, the sum and the products' sums in FP32.
#include "common.cuh"
#include "ptx.cuh"

namespace fp8bq {
namespace {

// A warp a query row; a lane has four neighbouring values of D.
__global__ void __launch_bounds__(128) prompt_attention_kernel(const PromptArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  if (row >= static_cast<int64_t>(a.T) * a.HQ) return;
  const int h = static_cast<int>(row % a.HQ), tok = static_cast<int>(row / a.HQ);
  auto bound = [&](int s) { return min(max(__ldg(a.offsets + s), 0), a.T); };
  int lo = 0, hi = a.S;  // the last s with offsets[s] <= tok
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (bound(mid) <= tok) lo = mid; else hi = mid;
  }
  const int start = bound(lo), end = bound(lo + 1);
  if (tok < start || tok >= end) return;
  const bool on = lane * 4 < a.D;
  auto load = [&](const uint16_t *p, float (&f)[4]) {
    uint2 v = make_uint2(0, 0);
    if (on) v = __ldg(reinterpret_cast<const uint2 *>(p + lane * 4));
    f[0] = __uint_as_float(v.x << 16), f[1] = __uint_as_float(v.x & 0xFFFF0000u);
    f[2] = __uint_as_float(v.y << 16), f[3] = __uint_as_float(v.y & 0xFFFF0000u);
  };
  float q[4], o[4] = {0, 0, 0, 0}, m = -INFINITY, l = 0.0f;
  load(a.q + tok * a.q_ts + h * a.q_hs, q);
  const int hk = h / (a.HQ / a.HK);
  for (int j = start; j <= tok; ++j) {
    float k[4], v[4];
    load(a.k + j * a.k_ts + hk * a.k_hs, k);
    load(a.v + j * a.v_ts + hk * a.v_hs, v);
    float s = q[0] * k[0] + q[1] * k[1] + q[2] * k[2] + q[3] * k[3];
#pragma unroll
    for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
    s *= a.scale_log2;
    const float mn = fmaxf(m, s), by = exp2f(m - mn), p = exp2f(s - mn);
    m = mn;
    l = l * by + p;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = o[i] * by + p * v[i];
  }
  if (!on) return;
  uint2 out;
  const float by = 1.0f / l;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(out.x) : "f"(o[1] * by), "f"(o[0] * by));
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(out.y) : "f"(o[3] * by), "f"(o[2] * by));
  *reinterpret_cast<uint2 *>(a.y + tok * a.y_ts + h * a.y_hs + lane * 4) = out;
}

}  // namespace

cudaError_t launch_prompt_attention(const PromptArgs &a, int num_sms, cudaStream_t st) {
  const int64_t rows = static_cast<int64_t>(a.T) * a.HQ;
  return launch_pdl(prompt_attention_kernel, dim3(static_cast<unsigned>((rows + 3) / 4)), dim3(128), 0,
                    st, a);
}

}  // namespace fp8bq
