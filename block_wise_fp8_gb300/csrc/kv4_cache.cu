// kv4_cache.cu -- rows written into the 4-bit paged cache, read back, and moved by
// weight (kv4.cuh has the layout).
//
// Writing: a group of 16 values has the scale
//   s = max(E4M3(min(amax / 6, 448)), 2^-9)         (binary32 division, nearest even)
// and the codes E2M1(x / s), the nearest of the exact quotient, ties to the even
// code, beyond 6 to 6; x is the BF16 value times RN(1 / g).  A NaN among the 16
// makes the scale NaN, so that it stays visible.
//
// Measured (8 heads of 128): 8192 tokens written and read back 23.1 us, over 12.8 at the
// copy rate; 32 sequences of up to 16384 tokens cut to 4096 by weight 192 us, of which the
// choice is 25, the move 46 and the read-back of what is kept the rest, over 117 in all.
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

// ---------------------------------------------------------------- append and read
//
// 4D bytes of rows and 9D/8 of a page a token and head.  HBM would be the floor; each of a
// token's D/4 threads looks its slot up and works its address out, so that a write, with
// the quotients, is bound by the ALU (73 %, issue slots 81 %) and a read by issue (67 %, at
// half the copy rate): 16.8 and 12.0 us cold for 8192 tokens x 8 heads x 128.  A thread
// has 8 values (half a group), so that rows, codes and scales are whole runs of a warp's
// lanes, and several tokens, whose loads are in flight together: 8192 tokens written and
// read back take 23.7, 24.0 and 24.8 us with 2, 3 and 4 to write (28.9 with 1 of each; whole
// groups a thread, one token of each: 24.8), 24.4 with 2 to read; 700000 rows read 210 and
// 198 with 2 and 4, 250 with 8 (with what goes before).  The quotients two at a time: 24.6
// -> 23.7.
constexpr int kAppendTokens = 2, kReadTokens = 4;

template <int D, int kRowTokens>
struct RowPlace {
  static constexpr int kLanes = D / 4;               // threads a token: keys, then values
  static constexpr int kTokens = kRowThreads / kLanes;  // tokens at a time
  int in, kv, piece;                                 // token of those, values?, run of 8 values
  __device__ RowPlace() : in(threadIdx.x / kLanes) {
    const int x = threadIdx.x % kLanes;
    kv = x >= D / 8;
    piece = x % (D / 8);
  }
  __device__ int64_t token(int u) const {
    return (static_cast<int64_t>(blockIdx.x) * kRowTokens + u) * kTokens + in;
  }
};

// RN(x / s) with r = RN(1 / s): one correction (Markstein).  No tie is moved, so that
// what is rounded to fewer bits next is the exact quotient's.
__device__ __forceinline__ float nearest_quotient(float x, float s, float r) {
  const float q = x * r;
  return __fmaf_rn(__fmaf_rn(-s, q, x), r, q);
}

template <int D>
__global__ void __launch_bounds__(kRowThreads) kv4_append_kernel(const Kv4AppendArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  const RowPlace<D, kAppendTokens> at;
  const int h = blockIdx.y;
  const Kv4Page p = kv4_page(1 << a.page_log2, D);
  const uint16_t *x = (at.kv ? a.v + h * a.v_hs : a.k + h * a.k_hs) + at.piece * 8;
  const int64_t ts = at.kv ? a.v_ts : a.k_ts;
  const float inv = at.kv ? a.v_inv : a.k_inv;
  Slot s[kAppendTokens];
  uint4 w[kAppendTokens];
#pragma unroll
  for (int u = 0; u < kAppendTokens; ++u) {
    const int64_t t = at.token(u);
    s[u].on = false;
    if (t < a.T) s[u] = slot_of(a.slots, a.slots64, t, a.pages, a.page_log2);
    w[u] = t < a.T ? __ldg(reinterpret_cast<const uint4 *>(x + t * ts)) : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int u = 0; u < kAppendTokens; ++u) {
    const uint32_t v[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
    // BF16 magnitudes are ordered as their bits are, infinity and then NaN on top
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) top = __vmaxu2(top, v[j] & 0x7FFF7FFFu);
    top = max(top & 0xFFFFu, top >> 16);
    top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
    const float amax = fminf(__uint_as_float(top << 16) * inv, 4096.0f);  // (over 6 * 448)
    uint32_t sb;  // RNE, saturating at 448
    asm("{\n\t.reg .b16 h;\n\tcvt.rn.satfinite.e4m3x2.f32 h, %1, %2;\n\tcvt.u32.u16 %0, h;\n\t}"
        : "=r"(sb)
        : "f"(0.0f), "f"(nearest_quotient(amax, kE2m1Max, 1.0f / kE2m1Max)));
    sb = max(sb & 0xFFu, 1u);
    const bool nan = top > 0x7F80u;
    if (nan) sb = kE4m3Nan;
    // the scale as binary32, and its reciprocal, correctly rounded after one Newton step
    // from the approximate one (for each of the 15 significands that a scale may have)
    const uint32_t e = sb >> 3, m = sb & 7u;
    const float sv = e ? __uint_as_float((e + 120u) << 23 | m << 20) : static_cast<float>(m) * kE4m3Least;
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(sv));
    r = __fmaf_rn(__fmaf_rn(-sv, r, 1.0f), r, r);
    // the quotients two at a time, as in nearest_quotient, of -x and -r: -0 stays -0
    const bool huge = __uint_as_float(top << 16) * inv > 4096.0f;
    const uint64_t minus_inv = pair(-inv, -inv), minus_r = pair(-r, -r), by = pair(sv, sv);
    uint32_t c = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint64_t y = mul2(pair(__uint_as_float(v[j] << 16), __uint_as_float(v[j] & 0xFFFF0000u)), minus_inv);
      if (huge) {  // infinities too
        float y0, y1;
        unpair(y, y0, y1);
        y = pair(fminf(fmaxf(y0, -4096.0f), 4096.0f), fminf(fmaxf(y1, -4096.0f), 4096.0f));
      }
      const uint64_t q = mul2(y, minus_r);
      float q0, q1;
      unpair(fma2(fma2(by, q, y), minus_r, q), q0, q1);
      uint32_t b;
      asm("{\n\t.reg .b8 p;\n\t.reg .b8 z;\n\tmov.b16 {z, p}, 0;\n\t"
          "cvt.rn.satfinite.e2m1x2.f32 p, %1, %2;\n\tmov.b32 %0, {p, z, z, z};\n\t}"
          : "=r"(b)
          : "f"(q1), "f"(q0));
      c |= b << (8 * j);
    }
    if (!s[u].on) continue;
    uint8_t *page = a.cache + (s[u].page * a.HK + h) * p.bytes;
    *reinterpret_cast<uint32_t *>(page + (at.kv ? p.v_codes : 0) + s[u].at * p.code_bytes + at.piece * 4) =
        nan ? 0u : c;
    if ((at.piece & 1) == 0)
      page[(at.kv ? p.v_scales : p.k_scales) + s[u].at * p.scale_bytes + at.piece / 2] = static_cast<uint8_t>(sb);
    if (a.weights && at.kv == 0 && at.piece == 0)
      a.weights[((s[u].page * a.HK + h) << a.page_log2) + s[u].at] = 0.0f;
  }
}

template <int D>
__global__ void __launch_bounds__(kRowThreads) kv4_read_kernel(const Kv4ReadArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  const RowPlace<D, kReadTokens> at;
  const int h = blockIdx.y;
  const Kv4Page p = kv4_page(1 << a.page_log2, D);
  uint16_t *y = (at.kv ? a.v + h * a.v_hs : a.k + h * a.k_hs) + at.piece * 8;
  const int64_t ts = at.kv ? a.v_ts : a.k_ts;
  const float gs = at.kv ? a.v_scale : a.k_scale;
  bool on[kReadTokens];
  uint32_t c[kReadTokens], sc[kReadTokens];
#pragma unroll
  for (int u = 0; u < kReadTokens; ++u) {
    const int64_t t = at.token(u);
    on[u] = false;
    if (t >= a.T) continue;
    const Slot s = slot_of(a.slots, a.slots64, t, a.pages, a.page_log2);
    on[u] = s.on;
    if (!s.on) continue;
    const uint8_t *page = a.cache + (s.page * a.HK + h) * p.bytes;
    c[u] = *reinterpret_cast<const uint32_t *>(page + (at.kv ? p.v_codes : 0) + s.at * p.code_bytes + at.piece * 4);
    sc[u] = page[(at.kv ? p.v_scales : p.k_scales) + s.at * p.scale_bytes + at.piece / 2];
  }
#pragma unroll
  for (int u = 0; u < kReadTokens; ++u) {
    if (!on[u]) continue;
    const uint32_t scale = both_low(e4m3x2_to_f16(sc[u]));
    uint32_t f[4], out[4];
    e2m1x8_to_f16(c[u], f);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float lo, hi;
      asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
          "cvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
          : "=f"(lo), "=f"(hi)
          : "r"(hmul2(f[j], scale)));
      unpair(mul2(pair(lo, hi), pair(gs, gs)), lo, hi);
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(out[j]) : "f"(hi), "f"(lo));
    }
    *reinterpret_cast<uint4 *>(y + at.token(u) * ts) = make_uint4(out[0], out[1], out[2], out[3]);
  }
}

// ---------------------------------------------------------------- evict: the choice

constexpr int kChooseThreads = 1024;
constexpr int kChooseWarps = kChooseThreads / 32;
constexpr int kBins = 2048;
constexpr int kBinCopies = 4;           // counts of every fourth lane: weights are close together
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
// order.  (Every token has its page, as the interface asks; one without counts as a
// NaN weight would, so that nothing is read out of range.)  Latency of one CTA: a
// gather of n weights, three counts, two walks (2203 tokens: 18 us with one warp
// looking for the bin, 64 bins a lane).
__global__ void __launch_bounds__(kChooseThreads) kv4_choose_kernel(const Kv4EvictArgs a) {
  extern __shared__ uint32_t keys[];
  __shared__ uint32_t bins[kBinCopies][kBins];
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
  if (cached) {
#pragma unroll 4
    for (int i = tid; i < m; i += kChooseThreads) keys[i] = key_at(i);
  }
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
      for (int i = tid; i < kBins * kBinCopies; i += kChooseThreads) (&bins[0][0])[i] = 0;
      __syncthreads();
      for (int i = tid; i < m; i += kChooseThreads) {
        const uint32_t k = key(i);
        if (pass == 0 || k >> high == prefix)
          atomicAdd(&bins[lane & (kBinCopies - 1)][k >> shift & ((1u << bits) - 1)], 1u);
      }
      __syncthreads();
      // from the top bin down, two a thread: how many lie above, up to the wanted one
      const int top = kBins - 1 - 2 * tid;
      uint32_t n0 = 0, n1 = 0;
#pragma unroll
      for (int c = 0; c < kBinCopies; ++c) n0 += bins[c][top], n1 += bins[c][top - 1];
      uint32_t upto = n0 + n1;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, upto, d);
        if (lane >= d) upto += v;
      }
      if (lane == 31) sums[0][warp] = upto;
      __syncthreads();
      upto += __reduce_add_sync(0xFFFFFFFFu, lane < warp ? sums[0][lane] : 0u);
      const uint32_t above = upto - n0 - n1;
      if (above < left && left <= upto) {  // one thread's
        const bool second = above + n0 < left;
        s_prefix = prefix << bits | static_cast<uint32_t>(top - second);
        s_left = left - above - (second ? n0 : 0u);
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

// A CTA moves kMoveRows kept tokens of a sequence and head: their old and new pages
// are looked up once, then the 16-byte words of codes, the scales and the weights go
// as whole runs of threads, several a thread in flight.  Bound by HBM: 2 x (9D/8 + 4)
// bytes a token (with all of a word's indexes worked out by its own thread, 32
// sequences of up to 4096 tokens x 8 heads took 104 us).
constexpr int kMoveRows = 128;
template <int D>
__global__ void __launch_bounds__(kRowThreads) kv4_move_kernel(const Kv4EvictArgs a) {
  __shared__ int64_t from[kMoveRows], to[kMoveRows];  // byte offsets of key codes, -1: none
  __shared__ int from_at[kMoveRows], to_at[kMoveRows];
  griddep_launch_dependents();
  griddep_wait();
  const int h = blockIdx.y, b = blockIdx.z, j0 = blockIdx.x * kMoveRows, tid = threadIdx.x;
  const int P = 1 << a.page_log2;
  const Kv4Page p = kv4_page(P, D);
  if (tid < kMoveRows) {
    const int j = j0 + tid;
    int64_t f = -1, t = -1;
    int fi = 0, ti = 0;
    if (j < a.budget) {
      const int k = a.kept[(static_cast<int64_t>(b) * a.HK + h) * a.budget + j];
      if (k >= 0) {
        const int src = __ldg(a.table + b * a.width + (k >> a.page_log2));
        const int dst = __ldg(a.new_table + b * a.new_width + (j >> a.page_log2));
        if (src >= 0 && src < a.pages && dst >= 0 && dst < a.pages) {
          f = (static_cast<int64_t>(src) * a.HK + h), t = (static_cast<int64_t>(dst) * a.HK + h);
          fi = k & (P - 1), ti = j & (P - 1);
          a.weights[(t << a.page_log2) + ti] = a.weights[(f << a.page_log2) + fi];
        }
      }
    }
    from[tid] = f < 0 ? -1 : f * p.bytes, to[tid] = t * p.bytes;
    from_at[tid] = fi, to_at[tid] = ti;
  }
  __syncthreads();
  constexpr int kWords = D / 16;  // 16-byte words of a token's codes, keys then values
  constexpr int kEach = kMoveRows * kWords / kRowThreads;
  uint4 w[kEach];
#pragma unroll
  for (int u = 0; u < kEach; ++u) {
    const int i = u * kRowThreads + tid, r = i / kWords, x = i % kWords, kv = x >= kWords / 2;
    if (from[r] >= 0)
      w[u] = *reinterpret_cast<const uint4 *>(a.cache + from[r] + (kv ? p.v_codes : 0) +
                                              from_at[r] * p.code_bytes + x % (kWords / 2) * 16);
  }
  // a token's scales, D/16 bytes of keys and of values: a thread each
  const int r = tid % kMoveRows, kv = tid / kMoveRows;
  uint32_t s[D / 64];
  if (from[r] >= 0) {
    const uint32_t *ss = reinterpret_cast<const uint32_t *>(
        a.cache + from[r] + (kv ? p.v_scales : p.k_scales) + from_at[r] * p.scale_bytes);
#pragma unroll
    for (int x = 0; x < D / 64; ++x) s[x] = ss[x];
  }
#pragma unroll
  for (int u = 0; u < kEach; ++u) {
    const int i = u * kRowThreads + tid, q = i / kWords, x = i % kWords, v = x >= kWords / 2;
    if (from[q] >= 0)
      *reinterpret_cast<uint4 *>(a.cache + to[q] + (v ? p.v_codes : 0) + to_at[q] * p.code_bytes +
                                 x % (kWords / 2) * 16) = w[u];
  }
  if (from[r] >= 0) {
    uint32_t *ds = reinterpret_cast<uint32_t *>(
        a.cache + to[r] + (kv ? p.v_scales : p.k_scales) + to_at[r] * p.scale_bytes);
#pragma unroll
    for (int x = 0; x < D / 64; ++x) ds[x] = s[x];
  }
}

// calls f(D as a constant)
template <typename F>
cudaError_t by_size(int D, F f) {
  return D == 64    ? f(std::integral_constant<int, 64>{})
         : D == 128 ? f(std::integral_constant<int, 128>{})
                    : f(std::integral_constant<int, 256>{});
}

unsigned blocks_of(int64_t n, int each) { return static_cast<unsigned>((n + each - 1) / each); }

}  // namespace

cudaError_t launch_kv4_append(const Kv4AppendArgs &a, cudaStream_t st) {
  return by_size(a.D, [&](auto d) {
    constexpr int D = decltype(d)::value;
    return launch_pdl(kv4_append_kernel<D>, dim3(blocks_of(a.T, kRowThreads / (D / 4) * kAppendTokens), a.HK),
                      dim3(kRowThreads), 0, st, a);
  });
}

cudaError_t launch_kv4_read(const Kv4ReadArgs &a, cudaStream_t st) {
  return by_size(a.D, [&](auto d) {
    constexpr int D = decltype(d)::value;
    return launch_pdl(kv4_read_kernel<D>, dim3(blocks_of(a.T, kRowThreads / (D / 4) * kReadTokens), a.HK),
                      dim3(kRowThreads), 0, st, a);
  });
}

cudaError_t launch_kv4_evict(const Kv4EvictArgs &a, cudaStream_t st) {
  cudaError_t e = allow_smem<kv4_choose_kernel>(kKeysCached * 4);
  if (e != cudaSuccess) return e;
  const int most = a.max_len - a.recent;  // keys of the longest sequence
  const size_t smem = static_cast<size_t>(most <= 0 ? 0 : most < kKeysCached ? most : kKeysCached) * 4;
  e = launch_pdl(kv4_choose_kernel, dim3(a.HK, a.B), dim3(kChooseThreads), smem, st, a);
  if (e != cudaSuccess) return e;
  return by_size(a.D, [&](auto d) {
    return launch_pdl(kv4_move_kernel<decltype(d)::value>, dim3(blocks_of(a.budget, kMoveRows), a.HK, a.B),
                      dim3(kRowThreads), 0, st, a);
  });
}

}  // namespace fp8bq
