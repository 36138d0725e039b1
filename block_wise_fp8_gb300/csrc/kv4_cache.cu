// kv4_cache.cu -- rows written into the 4-bit paged cache, read back, and moved by
// weight (kv4.cuh has the layout).
//
// Writing: a group of 16 values has the scale
//   s = max(E4M3(min(amax / 6, 448)), 2^-9)         (binary32 division, nearest even)
// and the codes E2M1(x / s), the nearest of the exact quotient, ties to the even
// code, beyond 6 to 6; x is the BF16 value times RN(1 / g).  A NaN among the 16
// makes the scale NaN, so that it stays visible.
#include "kv4.cuh"

namespace fp8bq {
namespace {

constexpr int kRowThreads = 256;

struct Slot {
  int64_t page;
  int at;
  bool on;
};

__device__ __forceinline__ Slot slot_of(const void *slots, int is64, int64_t t, int64_t pages,
                                        int page_log2) {
  const int64_t s = is64 ? __ldg(static_cast<const long long *>(slots) + t)
                         : static_cast<int64_t>(__ldg(static_cast<const int *>(slots) + t));
  Slot r;
  r.page = s >> page_log2;
  r.at = static_cast<int>(s & ((1 << page_log2) - 1));
  r.on = s >= 0 && r.page < pages;
  return r;
}

// ---------------------------------------------------------------- append

// A thread quantises one group: 32 bytes in, 8 bytes of codes and a scale out; a
// row's groups are neighbouring threads.  Bound by HBM (4D bytes a token and head
// in, 9D/8 out).
__global__ void __launch_bounds__(kRowThreads) kv4_append_kernel(const Kv4AppendArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  const int groups = a.D / 16;
  const int64_t per_token = static_cast<int64_t>(a.HK) * 2 * groups;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kRowThreads + threadIdx.x;
  const int64_t t = i / per_token;
  if (t >= a.T) return;
  const int in_token = static_cast<int>(i - t * per_token);
  const int g = in_token % groups, kv = in_token / groups % 2, h = in_token / groups / 2;
  const Slot s = slot_of(a.slots, a.slots64, t, a.pages, a.page_log2);
  if (!s.on) return;
  const uint16_t *x = (kv ? a.v + t * a.v_ts + h * a.v_hs : a.k + t * a.k_ts + h * a.k_hs) + g * 16;
  const float inv = kv ? a.v_inv : a.k_inv;
  uint32_t w[8];
  {
    const uint4 lo = __ldg(reinterpret_cast<const uint4 *>(x));
    const uint4 hi = __ldg(reinterpret_cast<const uint4 *>(x) + 1);
    w[0] = lo.x, w[1] = lo.y, w[2] = lo.z, w[3] = lo.w;
    w[4] = hi.x, w[5] = hi.y, w[6] = hi.z, w[7] = hi.w;
  }
  // BF16 magnitudes are ordered as their bits are, infinity and then NaN on top
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) top = __vmaxu2(top, w[j] & 0x7FFF7FFFu);
  top = max(top & 0xFFFFu, top >> 16);
  const float amax = __uint_as_float(top << 16) * inv;
  uint32_t sb;  // RNE, saturating at 448
  asm("{\n\t.reg .b16 h;\n\tcvt.rn.satfinite.e4m3x2.f32 h, %1, %2;\n\tcvt.u32.u16 %0, h;\n\t}"
      : "=r"(sb)
      : "f"(0.0f), "f"(__fdiv_rn(amax, kE2m1Max)));
  sb = max(sb & 0xFFu, 1u);
  const bool nan = top > 0x7F80u;
  if (nan) sb = kE4m3Nan;
  // the scale as binary32: four significant bits, so that q below is the nearest to
  // the exact quotient after one correction (Markstein), and no tie is moved
  const uint32_t e = sb >> 3, m = sb & 7u;
  const float sv = e ? __uint_as_float((e + 120u) << 23 | m << 20) : static_cast<float>(m) * kE4m3Least;
  const float r = __fdiv_rn(1.0f, sv);
  auto quotient = [&](float v) {
    v = fminf(fmaxf(v * inv, -4096.0f), 4096.0f);  // more than 6 * 448: infinities too
    const float q = v * r;
    return copysignf(__fmaf_rn(__fmaf_rn(-sv, q, v), r, q), v);  // -0 stays -0
  };
  uint32_t codes[2];
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    uint32_t c = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t two = w[half * 4 + j];
      uint32_t b;
      asm("{\n\t.reg .b8 p;\n\t.reg .b8 z;\n\tmov.b16 {z, p}, 0;\n\t"
          "cvt.rn.satfinite.e2m1x2.f32 p, %1, %2;\n\tmov.b32 %0, {p, z, z, z};\n\t}"
          : "=r"(b)
          : "f"(quotient(__uint_as_float(two & 0xFFFF0000u))), "f"(quotient(__uint_as_float(two << 16))));
      c |= b << (8 * j);
    }
    codes[half] = nan ? 0u : c;
  }
  const Kv4Page p = kv4_page(1 << a.page_log2, a.D);
  uint8_t *page = a.cache + (s.page * a.HK + h) * p.bytes;
  uint8_t *row = page + (kv ? p.v_codes : 0) + s.at * p.code_bytes;
  *reinterpret_cast<uint2 *>(row + g * 8) = make_uint2(codes[0], codes[1]);
  page[(kv ? p.v_scales : p.k_scales) + s.at * p.scale_bytes + g] = static_cast<uint8_t>(sb);
  if (a.weights && kv == 0 && g == 0)
    a.weights[((s.page * a.HK + h) << a.page_log2) + s.at] = 0.0f;
}

// ---------------------------------------------------------------- read

// A thread reads one group back: 9 bytes in, 32 out.
__global__ void __launch_bounds__(kRowThreads) kv4_read_kernel(const Kv4ReadArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  const int groups = a.D / 16;
  const int64_t per_token = static_cast<int64_t>(a.HK) * 2 * groups;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kRowThreads + threadIdx.x;
  const int64_t t = i / per_token;
  if (t >= a.T) return;
  const int in_token = static_cast<int>(i - t * per_token);
  const int g = in_token % groups, kv = in_token / groups % 2, h = in_token / groups / 2;
  const Slot s = slot_of(a.slots, a.slots64, t, a.pages, a.page_log2);
  if (!s.on) return;
  const Kv4Page p = kv4_page(1 << a.page_log2, a.D);
  const uint8_t *page = a.cache + (s.page * a.HK + h) * p.bytes;
  const uint2 c = *reinterpret_cast<const uint2 *>(page + (kv ? p.v_codes : 0) +
                                                   s.at * p.code_bytes + g * 8);
  const uint32_t sc =
      both_low(e4m3x2_to_f16(page[(kv ? p.v_scales : p.k_scales) + s.at * p.scale_bytes + g]));
  const float gs = kv ? a.v_scale : a.k_scale;
  uint32_t out[8];
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    uint32_t f[4];
    e2m1x8_to_f16(half ? c.y : c.x, f);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float lo, hi;
      asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
          "cvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
          : "=f"(lo), "=f"(hi)
          : "r"(hmul2(f[j], sc)));
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(out[half * 4 + j]) : "f"(hi * gs), "f"(lo * gs));
    }
  }
  uint16_t *y = (kv ? a.v + t * a.v_ts + h * a.v_hs : a.k + t * a.k_ts + h * a.k_hs) + g * 16;
  reinterpret_cast<uint4 *>(y)[0] = make_uint4(out[0], out[1], out[2], out[3]);
  reinterpret_cast<uint4 *>(y)[1] = make_uint4(out[4], out[5], out[6], out[7]);
}

// ---------------------------------------------------------------- evict: the choice

constexpr int kChooseThreads = 1024;
constexpr int kChooseWarps = kChooseThreads / 32;
constexpr int kBins = 2048;
constexpr int kKeysCached = 40 * 1024;  // keys kept in shared memory (160 KB)

// Weights in the order of whole numbers: NaN below everything, -0 as 0.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0u;
  const uint32_t b = __float_as_uint(w + 0.0f);
  return b >> 31 ? ~b : b | 0x80000000u;
}

// One CTA a sequence and head.  The heavy = budget - recent largest of the first
// m = n - recent weights: their smallest key by a radix selection (11 + 11 + 10
// bits), of the keys equal to it the first ones.  A warp then has a run of the
// tokens of its own, so that one exchange between the warps numbers them all in
// order.  Latency of one CTA: a gather of n weights, three counts, two walks.
__global__ void __launch_bounds__(kChooseThreads) kv4_choose_kernel(const Kv4EvictArgs a) {
  extern __shared__ uint32_t keys[];
  __shared__ uint32_t bins[kBins];
  __shared__ uint32_t sums[2][kChooseWarps];
  __shared__ uint32_t s_prefix, s_left;
  griddep_launch_dependents();
  griddep_wait();
  const int h = blockIdx.x, b = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int P = 1 << a.page_log2;
  const int n = min(max(__ldg(a.lens + b), 0), a.max_len);
  if (h == 0 && tid == 0) a.new_lens[b] = min(n, a.budget);
  int *kept = a.kept + (static_cast<int64_t>(b) * a.HK + h) * a.budget;
  if (n <= a.budget) {
    for (int i = tid; i < a.budget; i += kChooseThreads) kept[i] = i < n ? i : -1;
    return;
  }
  const int m = n - a.recent, heavy = a.budget - a.recent;
  const int *table = a.table + static_cast<int64_t>(b) * a.width;
  auto key_at = [&](int i) -> uint32_t {
    const int pg = __ldg(table + (i >> a.page_log2));
    if (pg < 0 || pg >= a.pages) return 0u;
    return weight_key(a.weights[((static_cast<int64_t>(pg) * a.HK + h) << a.page_log2) + (i & (P - 1))]);
  };
  const bool cached = m <= kKeysCached;
  if (cached)
    for (int i = tid; i < m; i += kChooseThreads) keys[i] = key_at(i);
  auto key = [&](int i) { return cached ? keys[i] : key_at(i); };
  // the key of the heavy-th largest, and how many of the keys equal to it are taken
  uint32_t prefix = 0, left = static_cast<uint32_t>(heavy);
  int shift = 32;
  if (heavy > 0) {
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int bits = pass == 2 ? 10 : 11;
      const int high = shift;  // bits above are settled
      shift -= bits;
      for (int i = tid; i < kBins; i += kChooseThreads) bins[i] = 0;
      __syncthreads();
      for (int i = tid; i < m; i += kChooseThreads) {
        const uint32_t k = key(i);
        if (pass == 0 || k >> high == prefix) atomicAdd(&bins[k >> shift & ((1u << bits) - 1)], 1u);
      }
      __syncthreads();
      if (warp == 0) {  // from the top: a lane has a run of bins
        const int per = (1 << bits) / 32;
        const int top = (1 << bits) - 1 - lane * per;
        uint32_t mine = 0;
        for (int j = 0; j < per; ++j) mine += bins[top - j];
        uint32_t upto = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, upto, d);
          if (lane >= d) upto += v;
        }
        uint32_t before = upto - mine;
        if (before < left && left <= upto) {
          int j = 0;
          while (before + bins[top - j] < left) before += bins[top - j++];
          s_prefix = prefix << bits | static_cast<uint32_t>(top - j);
          s_left = left - before;
        }
      }
      __syncthreads();
      prefix = s_prefix, left = s_left;
    }
  }
  // how many each warp's run keeps for sure, and how many equal the last key
  const int per_warp = ((m + kChooseWarps - 1) / kChooseWarps + 31) / 32 * 32;
  const int i0 = min(m, warp * per_warp), i1 = min(m, i0 + per_warp);
  uint32_t more = 0, same = 0;
  if (heavy > 0)
    for (int i = i0 + lane; i < i1; i += 32) {
      const uint32_t k = key(i);
      more += k > prefix, same += k == prefix;
    }
  more = __reduce_add_sync(0xFFFFFFFFu, more);
  same = __reduce_add_sync(0xFFFFFFFFu, same);
  if (lane == 0) sums[0][warp] = more, sums[1][warp] = same;
  __syncthreads();
  uint32_t at = 0, equal_before = 0;
  for (int w = 0; w < warp; ++w) at += sums[0][w], equal_before += sums[1][w];
  at += min(equal_before, left);
  if (heavy > 0)
    for (int base = i0; base < i1; base += 32) {
      const int i = base + lane;
      const uint32_t k = i < i1 ? key(i) : 0u;
      const bool is_same = i < i1 && k == prefix;
      const uint32_t eq = __ballot_sync(0xFFFFFFFFu, is_same);
      const uint32_t lower = (1u << lane) - 1u;
      const bool take = (i < i1 && k > prefix) || (is_same && equal_before + __popc(eq & lower) < left);
      const uint32_t got = __ballot_sync(0xFFFFFFFFu, take);
      if (take) kept[at + __popc(got & lower)] = i;
      at += __popc(got);
      equal_before += __popc(eq);
    }
  for (int i = tid; i < a.recent; i += kChooseThreads) kept[heavy + i] = m + i;
}

// ---------------------------------------------------------------- evict: the move

// D/16 threads a kept token and head, 16 bytes of codes each; the first of the keys'
// half also takes their scales, the first of the values' half theirs, the second
// thread the weight.
__global__ void __launch_bounds__(kRowThreads) kv4_move_kernel(const Kv4EvictArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  const int parts = a.D / 16;  // 16-byte words of a row's codes, keys then values
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kRowThreads + threadIdx.x;
  const int64_t row = i / parts;  // (b, h, place)
  if (row >= static_cast<int64_t>(a.B) * a.HK * a.budget) return;
  const int part = static_cast<int>(i - row * parts);
  const int j = static_cast<int>(row % a.budget);
  const int64_t bh = row / a.budget;
  const int h = static_cast<int>(bh % a.HK);
  const int64_t b = bh / a.HK;
  const int from = a.kept[row];
  if (from < 0) return;
  const int P = 1 << a.page_log2;
  const int src = __ldg(a.table + b * a.width + (from >> a.page_log2));
  const int dst = __ldg(a.new_table + b * a.new_width + (j >> a.page_log2));
  if (src < 0 || src >= a.pages || dst < 0 || dst >= a.pages) return;
  const Kv4Page p = kv4_page(P, a.D);
  const uint8_t *sp = a.cache + (static_cast<int64_t>(src) * a.HK + h) * p.bytes;
  uint8_t *dp = a.cache + (static_cast<int64_t>(dst) * a.HK + h) * p.bytes;
  const int si = from & (P - 1), di = j & (P - 1);
  const int half = parts / 2, kv = part >= half, word = part - kv * half;
  const int codes = kv ? p.v_codes : 0;
  *reinterpret_cast<uint4 *>(dp + codes + di * p.code_bytes + word * 16) =
      *reinterpret_cast<const uint4 *>(sp + codes + si * p.code_bytes + word * 16);
  if (word == 0) {
    const uint8_t *ss = sp + (kv ? p.v_scales : p.k_scales) + si * p.scale_bytes;
    uint8_t *ds = dp + (kv ? p.v_scales : p.k_scales) + di * p.scale_bytes;
    for (int w = 0; w < p.scale_bytes / 4; ++w)
      reinterpret_cast<uint32_t *>(ds)[w] = reinterpret_cast<const uint32_t *>(ss)[w];
  }
  if (part == 1)
    a.weights[((static_cast<int64_t>(dst) * a.HK + h) << a.page_log2) + di] =
        a.weights[((static_cast<int64_t>(src) * a.HK + h) << a.page_log2) + si];
}

unsigned blocks_of(int64_t threads) {
  return static_cast<unsigned>((threads + kRowThreads - 1) / kRowThreads);
}

}  // namespace

cudaError_t launch_kv4_append(const Kv4AppendArgs &a, cudaStream_t st) {
  return launch_pdl(kv4_append_kernel, dim3(blocks_of(a.T * a.HK * (a.D / 8))), dim3(kRowThreads), 0,
                    st, a);
}

cudaError_t launch_kv4_read(const Kv4ReadArgs &a, cudaStream_t st) {
  return launch_pdl(kv4_read_kernel, dim3(blocks_of(a.T * a.HK * (a.D / 8))), dim3(kRowThreads), 0,
                    st, a);
}

cudaError_t launch_kv4_evict(const Kv4EvictArgs &a, cudaStream_t st) {
  cudaError_t e = allow_smem<kv4_choose_kernel>(kKeysCached * 4);
  if (e != cudaSuccess) return e;
  const int most = a.max_len - a.recent;  // keys of the longest sequence
  const size_t smem = static_cast<size_t>(most <= 0 ? 0 : most < kKeysCached ? most : kKeysCached) * 4;
  e = launch_pdl(kv4_choose_kernel, dim3(a.HK, a.B), dim3(kChooseThreads), smem, st, a);
  if (e != cudaSuccess) return e;
  return launch_pdl(kv4_move_kernel,
                    dim3(blocks_of(static_cast<int64_t>(a.B) * a.HK * a.budget * (a.D / 16))),
                    dim3(kRowThreads), 0, st, a);
}

}  // namespace fp8bq
