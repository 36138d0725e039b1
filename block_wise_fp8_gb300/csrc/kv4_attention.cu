// kv4_attention.cu -- attention of a few new tokens of every sequence over its
// pages of the 4-bit cache (kv4.cuh has the layout).
//
// Per sequence, query token i, head h and its key/value head:
//   s_j = scale * g_k * q . k_j,  p_j = exp(s_j - max s) / sum exp(s - max s),
//   y = g_v * sum_j p_j v_j       over the cached tokens j that query i may see.
// The query rows of one key/value head (G heads x Tq tokens) share every key and
// value that is read, so they go through one pass over the pages: 9D/8 bytes a token
// and head, which is what bounds the kernel where contexts are long.
//
// Products by mma.sync m16n8k16 in FP16, whose fragments the codes are unpacked into
// from shared memory: the cache's rows are the wide side (16 tokens, or 16 of the D
// values), the query rows the narrow one (8).  code * scale is exact in FP16.  A
// query row is scaled by a power of two so that its largest value lies in [2^14,
// 2^15); what FP16 then drops lies 2^-39 below that.  p is rounded to FP16, 2^7 times as
// large as it is (half a step: 2^-11 of a p, 2^-32 of the largest), since the tokens
// beside one that draws nearly all of the weight may be what the row is made of; sums,
// maxima and the statistics are FP32.
//
// The order of the D values is free in the first product and that of the tokens in
// the second, so a lane takes D/4 neighbouring values of a key row, and D/8 of a
// value row, each lane's from one or two groups, with wide loads free of conflicts.
//
// Measured (64 heads over 8 of 128): 8 sequences of up to 131072 tokens 109 us, 0.71 of
// the copy rate; 64 of 512 to 8192 54 us, 0.58; one of 701 9.7 us.  Of a long run's time
// the issue slots are half busy and the ALU, which unpacks the codes, 46 %: latency of
// the three warps on a scheduler is what is left.  (Four groups of 112 registers and two
// stages, where three groups had 108 and 54.5, 10.0 and 13.3: 105 and 53.7, but 10.8, and
// 15.0 for 16 sequences of 1000.)
//
// Query rows an item: 8 up to 8 rows of a head, else 16, which share the unpacking.  16
// sequences of 6600 tokens, 16 rows: 56.8 us, as two items of 8 59.0; 64 rows: 158 and
// 200; one such sequence alone, which does not fill the device: 20.1 and 15.0.  The
// kernels of 16 rows with heads of 128 and 256 spill (184 and 188 bytes stored).
#include "kv4.cuh"

namespace fp8bq {
namespace {

constexpr int kWarps = 4;       // of a group

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

constexpr float kGrowth = 8.0f;  // log2: how far a score may pass a row's reference
constexpr float kLift = 7.0f;    // log2: p at the reference; p <= 2^15, which FP16 has room for

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

template <int D, int NB>
struct Sizes {
  static constexpr int kRows = 8 * NB;             // query rows of an item
  static constexpr int kMB = 2;                    // blocks of 16 tokens, a warp's of a tile
  static constexpr int kTile = kWarps * 16 * kMB;  // tokens a stage holds
  static constexpr int kStages = D == 64 ? 4 : D == 128 && NB == 1 ? 3 : 2;
  static constexpr int kKvBytes = kTile * 9 * D / 8;
  static constexpr int kStageBytes = kKvBytes + kRows * D * 2;  // and an item's query rows
  static constexpr int kPart = kRows * (D + 3);    // floats of a group's part of an item
  // three quarters of every warp's sums, and all rows' maxima and sums
  static constexpr int kJoinBytes = 3 * kRows * D * 4 + kWarps * kRows * 8;
  static constexpr int kGroupBytes = kStages * kStageBytes + kJoinBytes;
  // Groups of warps that work for themselves, and one more for the copies, which leaves
  // its registers to them: 160 a thread, three warps on a scheduler.  (Three CTAs of four
  // warps and a copying one: 128; two: 168.  16 sequences of 6600 tokens, 64 heads over
  // 8, eight new tokens each: 156 us, with two such CTAs 180; with one new token 36 and
  // with three such CTAs 37.)
  static constexpr int kGroups = D <= 128 ? 3 : NB == 1 ? 2 : 1;
  static constexpr int kThreads = (kGroups + 1) * 128;
  static constexpr int kRegs = kGroups == 3 ? 160 : 232, kCopyRegs = kGroups == 3 ? 32 : 40;
  static constexpr int kSmem = kGroups * kGroupBytes;  // and (B + 1) * 4
};

// Where a group is in the flattened list of slots: sequence, item of it, slot of the
// item (its tiles first).
struct Place {
  int b, item, tile, tiles;  // tiles: of each of the sequence's items
};

struct Bars {
  uint64_t full[4], empty[4];
  uint32_t abort, ticket[2];
  uint32_t pages[4];  // which pages of a stage's tile are there
};

// The work of the batch as a list of slots: an item's tiles, and kJoinSlots more for
// what an item costs besides (its queries, the join of the warps' sums).  first[b]
// counts those of one item of each sequence before b.  Every group takes an equal run
// of the whole list (the first `more` of them one slot more), so that ragged batches
// fill the device evenly (64 sequences of 512 to 8192 tokens, 64 heads over 8: 61.5 us
// with no slots for the joins, 56.7, 55.2, 55.5 and 57.0 with one to four).
constexpr int kJoinSlots = 2;
struct Plan {
  const int *first;  // [B + 1]
  int B, items;      // items a sequence: HK * blocks
  int each, more;    // slots a group, and groups with one more
  __device__ Plan(const int *f, int B_, int items_, int most, int least) : first(f), B(B_), items(items_) {
    const int total = f[B_] * items_;
    // fewer groups than there are take part where there are few slots: at least `least`
    // each, since a part costs as much as a tile to add to the others'.  With 8 rows an
    // item two (one sequence of 8192 tokens, 64 heads over 8: 18.0, 14.1, 14.2 and 13.4 us
    // with 1 to 4; of 701: 10.2, 10.1, 10.6 and 11.2), with 16, whose parts are twice as
    // large, three (two of 6600, four tokens each, 32 heads: 26.4, 24.1, 22.5 and 23.3)
    const int active = min((max(total, 1) + least - 1) / least, most);
    each = total / active;
    more = total - each * active;
  }
  __device__ int total() const { return first[B] * items; }
  __device__ int start(int group) const { return min(total(), group * each + min(group, more)); }
  __device__ int group_of(int slot) const {
    const int longer = more * (each + 1);
    return slot < longer ? slot / (each + 1) : more + (slot - longer) / each;
  }
  __device__ Place at(int f) const {
    int lo = 0, hi = B;  // the last b with first[b] * items <= f, which has slots
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (first[mid] * items <= f) lo = mid; else hi = mid;
    }
    Place p;
    p.b = lo;
    const int slots = first[lo + 1] - first[lo], in = f - first[lo] * items;
    p.tiles = slots - kJoinSlots;
    p.item = in / slots;
    p.tile = in - p.item * slots;
    return p;
  }
  __device__ void next(Place &p) const {
    if (++p.tile < p.tiles + kJoinSlots) return;
    p.tile = 0;
    if (++p.item < items) return;
    p.item = 0;
    do {
      ++p.b;
    } while (p.b < B && first[p.b + 1] == first[p.b]);
    if (p.b < B) p.tiles = first[p.b + 1] - first[p.b] - kJoinSlots;
  }
};

template <int D, int NB>
__global__ void __launch_bounds__(Sizes<D, NB>::kThreads, 1) kv4_attention_kernel(const Kv4AttnArgs a) {
  using S = Sizes<D, NB>;
  constexpr int kRows = S::kRows, kStages = S::kStages, kMB = S::kMB, kTile = S::kTile;
  constexpr int kKeyWords = D / 32;       // 32-bit words of codes a lane takes of a key row
  constexpr int kTiles = D / 16;          // products of 16 values of the D
  constexpr int kValueWords = D / 64;     // words of codes a lane takes of a value row
  constexpr int kQuarter = kTiles / kWarps;
  constexpr int kGroups = S::kGroups, kThreads = S::kThreads;
  extern __shared__ __align__(128) uint8_t all_smem[];
  int *first = reinterpret_cast<int *>(all_smem + S::kSmem);
  __shared__ Bars all_bars[kGroups];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5 & 3;  // of its group
  // the last group of warps has a copying warp for each of the others
  const bool copies = threadIdx.x >= kGroups * 128;
  const int group = copies ? warp : threadIdx.x >> 7;
  // what a group has as its number: neighbours are on different SMs, for when there is
  // less work than groups
  const int me = group * gridDim.x + blockIdx.x, everyone = kGroups * gridDim.x;
  if (threadIdx.x < kGroups) {
    Bars &b = all_bars[threadIdx.x];
    for (int i = 0; i < kStages; ++i) mbar_init(&b.full[i], 1), mbar_init(&b.empty[i], kWarps);
    b.abort = 0;
    fence_mbar_init();
  }
  griddep_launch_dependents();
  griddep_wait();
  const int P = 1 << a.page_log2;
  const int R = a.G * a.Tq, blocks = (R + kRows - 1) / kRows;
  const Kv4Page pg = kv4_page(P, D);
  auto length = [&](int b) { return min(max(__ldg(a.lens + b), 0), a.max_len); };
  for (int b = threadIdx.x; b < a.B; b += kThreads) {
    const int tiles = (length(b) + kTile - 1) / kTile;
    first[b + 1] = tiles ? tiles + kJoinSlots : 0;
  }
  if (threadIdx.x == 0) first[0] = 0;
  __syncthreads();
  if (threadIdx.x < 32) {
    int run = 0;
    for (int b0 = 0; b0 < a.B; b0 += 32) {
      int v = b0 + lane < a.B ? first[b0 + lane + 1] : 0;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int u = __shfl_up_sync(0xFFFFFFFFu, v, d);
        if (lane >= d) v += u;
      }
      v += run;
      if (b0 + lane < a.B) first[b0 + lane + 1] = v;
      run = __shfl_sync(0xFFFFFFFFu, v, 31);
    }
  }
  __syncthreads();
  if (copies) {
    if constexpr (kGroups > 1) setmaxnreg_dec<S::kCopyRegs>();
    // (the group's warps beyond the others' number have no run: the list ends before it)
    const Plan plan(first, a.B, a.HK * blocks, everyone, NB + 1);
    const int f0 = plan.start(me), f1 = plan.start(me + 1);
    Bars &bars = all_bars[min(group, kGroups - 1)];
    volatile uint32_t *abort = &bars.abort;
    uint8_t *smem = all_smem + group * S::kGroupBytes;
    // ---- copies: a tile's pages, each one run of bytes, into the stage, and with an
    // item's first tile its query rows
    Place p = f0 < f1 ? plan.at(f0) : Place{};
    const int per_tile = kTile >> a.page_log2;
    auto look_up = [&]() -> int {  // this lane's page of tile p, -1 where there is none
      const int at = p.tile * per_tile + lane;
      if (p.tile >= p.tiles || lane >= per_tile || (at << a.page_log2) >= length(p.b)) return -1;
      const int page = __ldg(a.table + static_cast<int64_t>(p.b) * a.width + at);
      return page < a.pages ? page : -1;
    };
    int page = f0 < f1 ? look_up() : -1;
    int st = 0, ph = 1, filled = 0;
    for (int f = f0; f < f1; ++f) {
      if (p.tile >= p.tiles) {
        plan.next(p);
        if (f + 1 < f1) page = look_up();
        continue;
      }
      const int head = p.item / blocks, row = (p.item - head * blocks) * kRows + lane;
      const bool q_too = f == f0 || p.tile == 0;
      const bool q_on = q_too && lane < kRows && row < R;
      if (!__all_sync(0xFFFFFFFFu, mbar_wait(&bars.empty[st], ph, abort, a.wait_limit_ns))) break;
      const bool on = page >= 0;
      const uint32_t there = __ballot_sync(0xFFFFFFFFu, on);
      if (lane == 0) {
        bars.pages[st] = there;
        const int rows = q_too ? min(kRows, R - row) : 0;  // (row: the item's first)
        mbar_arrive_expect_tx(&bars.full[st], __popc(there) * pg.bytes + rows * D * 2);
      }
      __syncwarp();
      if (q_on) {
        const int i = row / a.G;
        bulk_load_1d(smem + st * S::kStageBytes + S::kKvBytes + lane * D * 2,
                     a.q + (static_cast<int64_t>(p.b) * a.Tq + i) * a.q_ts +
                         static_cast<int64_t>(head * a.G + row - i * a.G) * a.q_hs,
                     D * 2, &bars.full[st]);
      }
      if (on && !(a.fault && me == 0 && filled == 0))
        bulk_load_1d(smem + st * S::kStageBytes + lane * pg.bytes,
                     a.cache + (static_cast<int64_t>(page) * a.HK + head) * pg.bytes, pg.bytes,
                     &bars.full[st]);
      if (++st == kStages) st = 0, ph ^= 1;
      ++filled;
      plan.next(p);
      if (f + 1 < f1) page = look_up();
    }
    // copies in flight land before the memory is given up, also those that nobody waits for
    // any more: the group may give up at any time, after the last copy too
    for (int k = max(filled - kStages, 0); k < filled; ++k)
      mbar_wait_alone(&bars.full[k % kStages], k / kStages & 1, a.wait_limit_ns);
  } else {
    if constexpr (kGroups > 1) setmaxnreg_inc<S::kRegs>();
    const Plan plan(first, a.B, a.HK * blocks, everyone, NB + 1);
    const int f0 = plan.start(me), f1 = plan.start(me + 1);
    const int tid = threadIdx.x & 127;  // of the group
    Bars &bars = all_bars[group];
    volatile uint32_t *abort = &bars.abort;
    uint8_t *smem = all_smem + group * S::kGroupBytes;
    float4 *join = reinterpret_cast<float4 *>(smem + kStages * S::kStageBytes);
    float2 *join_stat = reinterpret_cast<float2 *>(join + 3 * kRows * D / 4);
    auto meet = [&] { named_bar_sync(1 + group, kWarps * 32); };  // the group's warps
    const int g = lane >> 2, t = lane & 3;
    // tokens of a block of 16 as the products' rows take them
    const int key_row = (g >> 1) + (g & 1) * 4;
    uint32_t qf[kTiles][NB][2];   // the query rows, a value pair a register
    float qs[NB][2];              // log2 units a product, of this lane's two columns
    float mx[NB][2], sum[NB][2];
    float o[kTiles][NB][4];
    int ends[NB][2];              // tokens that the column's query may see
    int st = 0, ph = 0;
    Place p = f0 < f1 ? plan.at(f0) : Place{};
    int len = 0, row0 = 0, head = 0;
    Place early = p, late = p;    // items with parts elsewhere: before this run, behind it
    bool has_early = false, has_late = false;
    // what a part with maximum m counts under the maximum of all (one with nothing seen
    // holds zeros, or the NaN that a row was given).  Maxima are kept as they come out of
    // the products, as within a warp: all parts of a row have its scale in common, and the
    // scaled ones may pass FP32's range, or differ by less than their last place.
    auto factor = [](float m, float all, float by) {
      const float d = m == all ? 0.0f : m - all;  // (both may be -inf)
      return ex2(d * by);
    };
    // product j of query rows nb * 8 + 2t, + 1 of an item: two values of each
    auto finish = [&](int b, int hd, int r0, int nb, int j, float4 v, const float (&m)[2], const float (&l)[2],
                      const float (&qb)[NB][2]) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int r = r0 + nb * 8 + 2 * t + c;
        if (r >= R) continue;
        const int i = r / a.G;
        const float by = l[c] == 0.0f ? 0.0f : a.v_scale / l[c];
        uint32_t out;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(out) : "f"((c ? v.w : v.z) * by), "f"((c ? v.y : v.x) * by));
        *reinterpret_cast<uint32_t *>(a.y + (static_cast<int64_t>(b) * a.Tq + i) * a.y_ts +
                                      static_cast<int64_t>(hd * a.G + r - i * a.G) * a.y_hs +
                                      g * (D / 8) + 2 * j) = out;
        if (a.stats && j == 0 && g == 0)
          *reinterpret_cast<float4 *>(a.stats + ((static_cast<int64_t>(b) * a.HK + hd) * R + r) * 4) =
              make_float4(m[c], qb[nb][c], l[c], 0.0f);
      }
    };
    // The warps' sums together, put(query rows nb, product j, its sums, maxima, sums of
    // p): every warp has sums of the same values in the same places, and ends up with a
    // quarter of them.
    auto together = [&](const float (&m)[NB][2], const float (&l)[NB][2], const float (&qb)[NB][2],
                        auto &&put) {
      meet();  // what the memory held before has been read
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
        for (int c = 0; c < 2; ++c)
          if (g == 0) join_stat[warp * kRows + nb * 8 + 2 * t + c] = make_float2(m[nb][c], l[nb][c]);
#pragma unroll
        for (int j = 0; j < kTiles; ++j) {
          const int to = j / kQuarter, from = warp - (warp > to);  // place among the other three
          if (to != warp)
            join[((j * NB + nb) * 3 + from) * 32 + lane] =
                make_float4(o[j][nb][0], o[j][nb][1], o[j][nb][2], o[j][nb][3]);
        }
      }
      meet();
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        float ma[2], la[2], by[kWarps][2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float2 st2[kWarps];
          ma[c] = -INFINITY, la[c] = 0.0f;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) {
            st2[w] = join_stat[w * kRows + nb * 8 + 2 * t + c];
            ma[c] = fmaxf(ma[c], st2[w].x);
          }
#pragma unroll
          for (int w = 0; w < kWarps; ++w) {
            by[w][c] = factor(st2[w].x, ma[c], qb[nb][c]);
            la[c] += st2[w].y * by[w][c];
          }
        }
#pragma unroll
        for (int k = 0; k < kQuarter; ++k) {
          float4 v = make_float4(0, 0, 0, 0);
#pragma unroll
          for (int w = 0; w < kWarps; ++w) {  // the warps in order, whoever sums
            float4 x;
            if (w == warp) {
#pragma unroll
              for (int q = 0; q < kWarps; ++q)
                if (q == warp)
                  x = make_float4(o[q * kQuarter + k][nb][0], o[q * kQuarter + k][nb][1],
                                  o[q * kQuarter + k][nb][2], o[q * kQuarter + k][nb][3]);
            } else {
              x = join[(((warp * kQuarter + k) * NB + nb) * 3 + w - (w > warp)) * 32 + lane];
            }
            v.x += x.x * by[w][0], v.y += x.y * by[w][1], v.z += x.z * by[w][0], v.w += x.w * by[w][1];
          }
          put(nb, warp * kQuarter + k, v, ma, la);
        }
      }
    };
    for (int f = f0; f < f1; ++f, plan.next(p)) {
      if (p.tile >= p.tiles) continue;
      // (after a wait that gave up the walk goes on, over whatever the memory holds,
      // so that no warp leaves the others at a barrier)
      mbar_wait(&bars.full[st], ph, abort, a.wait_limit_ns);
      const uint8_t *stage = smem + st * S::kStageBytes;
      if (f == f0 || p.tile == 0) {
        // ---- a new item: its query rows
        len = length(p.b);
        head = p.item / blocks;
        row0 = (p.item - head * blocks) * kRows;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          const int row = row0 + nb * 8 + g;
          uint4 raw[D / 32];
          uint32_t top = 0;
#pragma unroll
          for (int i = 0; i < D / 32; ++i) raw[i] = make_uint4(0, 0, 0, 0);
          if (row < R) {
            const uint4 *q = reinterpret_cast<const uint4 *>(stage + S::kKvBytes + (nb * 8 + g) * D * 2 + t * (D / 2));
#pragma unroll
            for (int k = 0; k < D / 32; ++k) raw[k] = q[k];
          }
#pragma unroll
          for (int i = 0; i < D / 32; ++i)
            top = __vmaxu2(top, __vmaxu2(__vmaxu2(raw[i].x & 0x7FFF7FFFu, raw[i].y & 0x7FFF7FFFu),
                                         __vmaxu2(raw[i].z & 0x7FFF7FFFu, raw[i].w & 0x7FFF7FFFu)));
          top = max(top & 0xFFFFu, top >> 16);
          top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
          top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
          // the row's power of two: its largest value to [2^14, 2^15)
          const int e = top >> 7;
          const int up = e == 255 ? 0 : 14 + 127 - max(e, 24);
          const float by = __uint_as_float(static_cast<uint32_t>(127 + up) << 23);
          // (never 0: -inf times it has to stay -inf; nor infinite: 0 times it has to stay 0)
          const float back = fminf(
              fmaxf(__uint_as_float(static_cast<uint32_t>(127 - up) << 23) * a.scale_log2, 1.2e-38f), 3.4e38f);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            qs[nb][c] = __shfl_sync(0xFFFFFFFFu, back, (2 * t + c) * 4);
            const int r = row0 + nb * 8 + 2 * t + c;
            ends[nb][c] = r < R ? len - (a.Tq - 1 - r / a.G) : len;
            mx[nb][c] = -INFINITY, sum[nb][c] = 0.0f;
          }
#pragma unroll
          for (int i = 0; i < D / 32; ++i) {
            const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
              qf[i * 2 + j / 2][nb][j & 1] = pack_f16(__uint_as_float(w[j] << 16) * by,
                                                      __uint_as_float(w[j] & 0xFFFF0000u) * by);
          }
#pragma unroll
          for (int j = 0; j < kTiles; ++j)
#pragma unroll
            for (int c = 0; c < 4; ++c) o[j][nb][c] = 0.0f;
        }
      }
      const int tok0 = p.tile * kTile + warp * (16 * kMB);
      const uint32_t there = bars.pages[st];
      const int per_tile = kTile >> a.page_log2;
      // every token of the warp's seen by every row, and the pages there
      const int seen_by_all = len - (a.Tq - 1);
      const bool whole = __all_sync(
          0xFFFFFFFFu, tok0 + 16 * kMB <= seen_by_all && there == (1u << per_tile) - 1u);
      auto block_of = [&](int mb, int &in) {  // page of the warp's 16-token block, place in it
        const int at = (warp * kMB + mb) * 16;
        in = at & (P - 1);
        return stage + (at >> a.page_log2) * pg.bytes;
      };
      if (whole || tok0 < len) {
        float s[kMB][NB][4];
        // ---- scores
#pragma unroll
        for (int mb = 0; mb < kMB; ++mb) {
          int in;
          const uint8_t *page = block_of(mb, in);
          uint32_t w[2][kKeyWords];
          uint32_t sc[2][D / 64];  // a group's scale in both halves
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const int row = in + key_row + r * 8;
            const uint8_t *codes = page + row * (D / 2) + t * (D / 8);
            if constexpr (D == 64) {
              const uint2 v = *reinterpret_cast<const uint2 *>(codes);
              w[r][0] = v.x, w[r][1] = v.y;
            } else {
#pragma unroll
              for (int i = 0; i < D / 128; ++i) {
                const uint4 v = reinterpret_cast<const uint4 *>(codes)[i];
                w[r][i * 4] = v.x, w[r][i * 4 + 1] = v.y, w[r][i * 4 + 2] = v.z, w[r][i * 4 + 3] = v.w;
              }
            }
            const uint8_t *scales = page + pg.k_scales + row * (D / 16) + t * (D / 64);
            if constexpr (D == 64) {
              sc[r][0] = both_low(e4m3x2_to_f16(*scales));
            } else {
#pragma unroll
              for (int i = 0; i < D / 128; ++i) {
                const uint32_t two = e4m3x2_to_f16(reinterpret_cast<const uint16_t *>(scales)[i]);
                sc[r][2 * i] = both_low(two), sc[r][2 * i + 1] = both_high(two);
              }
            }
          }
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int c = 0; c < 4; ++c) s[mb][nb][c] = 0.0f;
#pragma unroll
          for (int i = 0; i < kKeyWords; ++i) {
            uint32_t lo[4], hi[4];
            e2m1x8_to_f16(w[0][i], lo);
            e2m1x8_to_f16(w[1][i], hi);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const uint32_t f[4] = {hmul2(lo[2 * k], sc[0][i / 2]), hmul2(hi[2 * k], sc[1][i / 2]),
                                     hmul2(lo[2 * k + 1], sc[0][i / 2]), hmul2(hi[2 * k + 1], sc[1][i / 2])};
#pragma unroll
              for (int nb = 0; nb < NB; ++nb) mma_f16(s[mb][nb], f, qf[2 * i + k][nb][0], qf[2 * i + k][nb][1]);
            }
          }
        }
        // ---- what a row may not see goes to -inf
        if (!whole) {
#pragma unroll
          for (int mb = 0; mb < kMB; ++mb) {
            const bool here = there >> ((warp * kMB + mb) * 16 >> a.page_log2) & 1u;
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                const int tok = tok0 + mb * 16 + key_row + (c >> 1) * 8;
                if (!here || tok >= ends[nb][c & 1]) s[mb][nb][c] = -INFINITY;
              }
          }
        }
        if (a.logits) {
          float *row = a.logits + ((static_cast<int64_t>(p.b) * a.HK + head) * R + row0 + 2 * t) * a.max_len + tok0 + key_row;
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              if (row0 + nb * 8 + 2 * t + c >= R) continue;
              float *at = row + static_cast<int64_t>(nb * 8 + c) * a.max_len;
#pragma unroll
              for (int mb = 0; mb < kMB; ++mb)
#pragma unroll
                for (int half = 0; half < 2; ++half)
                  if (whole || tok0 + key_row + mb * 16 + half * 8 < a.max_len)
                    at[mb * 16 + half * 8] = s[mb][nb][half * 2 + c];
            }
        }
        // ---- the reference that p is held to: a score of the row that no other has
        // passed by more than 8 in log2 units; what was summed follows it.
        // (The difference is taken before the scale, so that it is exact where it is
        // small, however large the scores are.)
        bool grew = false;
        float lm[NB][2];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            lm[nb][c] = fmaxf(s[0][nb][c], s[0][nb][c + 2]);
#pragma unroll
            for (int mb = 1; mb < kMB; ++mb) lm[nb][c] = fmaxf(lm[nb][c], fmaxf(s[mb][nb][c], s[mb][nb][c + 2]));
            grew |= (lm[nb][c] - mx[nb][c]) * qs[nb][c] > kGrowth;
          }
        if (__any_sync(0xFFFFFFFFu, grew)) {
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            float fix[2];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              float m = lm[nb][c];
              m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 4));
              m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 8));
              m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 16));
              const bool up = (m - mx[nb][c]) * qs[nb][c] > kGrowth;
              fix[c] = up ? ex2((mx[nb][c] - m) * qs[nb][c]) : 1.0f;
              if (up) mx[nb][c] = m;
              sum[nb][c] *= fix[c];
            }
#pragma unroll
            for (int j = 0; j < kTiles; ++j)
#pragma unroll
              for (int c = 0; c < 4; ++c) o[j][nb][c] *= fix[c & 1];
          }
        }
        // ---- p, and its fragments for the second product: rows become columns
        uint32_t pf[kMB][NB][2];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          // (a row that has seen nothing: -inf - 0)
          const uint64_t ref = pair(mx[nb][0] == -INFINITY ? 0.0f : -mx[nb][0],
                                    mx[nb][1] == -INFINITY ? 0.0f : -mx[nb][1]);
          const uint64_t by = pair(qs[nb][0], qs[nb][1]);
#pragma unroll
          for (int mb = 0; mb < kMB; ++mb) {
            float p0, p1, p2, p3;
            unpair(fma2(add2(pair(s[mb][nb][0], s[mb][nb][1]), ref), by, pair(kLift, kLift)), p0, p1);
            unpair(fma2(add2(pair(s[mb][nb][2], s[mb][nb][3]), ref), by, pair(kLift, kLift)), p2, p3);
            p0 = ex2(p0), p1 = ex2(p1), p2 = ex2(p2), p3 = ex2(p3);
            sum[nb][0] += p0 + p2, sum[nb][1] += p1 + p3;
            pf[mb][nb][0] = transpose8x8(pack_f16(p0, p1));
            pf[mb][nb][1] = transpose8x8(pack_f16(p2, p3));
          }
        }
        // ---- p times the values.  Those of tokens that no row may see count as 0,
        // whatever their bytes hold; a NaN that some rows see goes to those rows alone.
        auto seen_scales = [&](uint32_t b, int r, int mb) -> uint32_t {
          const bool here = there >> ((warp * kMB + mb) * 16 >> a.page_log2) & 1u;
          const int base = tok0 + mb * 16 + r * 8, tok = base + key_row;
          if (!here || tok >= len) b = 0;
#pragma unroll
          for (int k = 0; k < D / 64; ++k) {
            const bool bad = (b >> (8 * k) & 0x7Fu) == kE4m3Nan && tok >= seen_by_all;
            if (bad) b &= ~(0xFFu << (8 * k));
            for (uint32_t who = __ballot_sync(0xFFFFFFFFu, bad); who; who &= who - 1) {
              const int from = __ffs(who) - 1, fg = from >> 2;
              const int group = (from & 3) * (D / 64) + k, other = base + (fg >> 1) + (fg & 1) * 4;
              // this lane's values are D/8 from g * D/8 on
              constexpr int kPer = D == 256 ? 2 : 1;
#pragma unroll
              for (int w = 0; w < kPer; ++w) {
                if (group != (D == 64 ? g >> 1 : g * kPer + w)) continue;
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                  for (int c = 0; c < 2; ++c)
                    if (other < ends[nb][c])
#pragma unroll
                      for (int j = w * (kTiles / kPer); j < (w + 1) * (kTiles / kPer); ++j)
                        o[j][nb][c] = o[j][nb][c + 2] = NAN;
              }
            }
          }
          return b;
        };
#pragma unroll
        for (int mb = 0; mb < kMB; ++mb) {
          int in;
          const uint8_t *page = block_of(mb, in);
          uint32_t w[4][kValueWords];  // tokens 2t, 2t+1, 2t+8, 2t+9 of the products' order
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int row = in + t + r * 4;
            const uint8_t *codes = page + pg.v_codes + row * (D / 2) + g * (D / 16);
            if constexpr (D == 64) {
              w[r][0] = *reinterpret_cast<const uint32_t *>(codes);
            } else if constexpr (D == 128) {
              const uint2 v = *reinterpret_cast<const uint2 *>(codes);
              w[r][0] = v.x, w[r][1] = v.y;
            } else {
              const uint4 v = *reinterpret_cast<const uint4 *>(codes);
              w[r][0] = v.x, w[r][1] = v.y, w[r][2] = v.z, w[r][3] = v.w;
            }
          }
          // the tokens' scales: a lane has those of one of 8 tokens for two columns of
          // lanes (its own of the key scales' pattern), and gets those of two tokens for
          // its own by a transposition
          constexpr int kScales = D == 256 ? 2 : 1;
          uint32_t sv[2][kScales];  // of tokens 2t, 2t+1 | 2t+8, 2t+9
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const int row = in + key_row + r * 8;
            const uint8_t *scales = page + pg.v_scales + row * (D / 16) + t * (D / 64);
            uint32_t b = D == 64    ? *scales
                         : D == 128 ? *reinterpret_cast<const uint16_t *>(scales)
                                    : *reinterpret_cast<const uint32_t *>(scales);
            if (!whole) b = seen_scales(b, r, mb);
            if constexpr (D == 64) {
              sv[r][0] = transpose8x8(both_low(e4m3x2_to_f16(b)));
            } else if constexpr (D == 128) {
              sv[r][0] = transpose8x8(e4m3x2_to_f16(b));
            } else {
              const uint32_t lo = e4m3x2_to_f16(b & 0xFFFFu), hi = e4m3x2_to_f16(b >> 16);
              sv[r][0] = transpose8x8(__byte_perm(lo, hi, 0x5410));
              sv[r][1] = transpose8x8(__byte_perm(lo, hi, 0x7632));
            }
          }
#pragma unroll
          for (int i = 0; i < kValueWords; ++i) {
            // the codes of two tokens side by side: even values, odd values
            uint32_t ev[2][4], od[2][4];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const uint32_t x = w[2 * k][i], y = w[2 * k + 1][i];
              e2m1x8_to_f16((x & 0x0F0F0F0Fu) | (y << 4 & 0xF0F0F0F0u), ev[k]);
              e2m1x8_to_f16((x >> 4 & 0x0F0F0F0Fu) | (y & 0xF0F0F0F0u), od[k]);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int group = D == 256 ? i / 2 : 0;
              const uint32_t f[4] = {hmul2(ev[0][j], sv[0][group]), hmul2(od[0][j], sv[0][group]),
                                     hmul2(ev[1][j], sv[1][group]), hmul2(od[1][j], sv[1][group])};
#pragma unroll
              for (int nb = 0; nb < NB; ++nb) mma_f16(o[i * 4 + j][nb], f, pf[mb][nb][0], pf[mb][nb][1]);
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.empty[st]);
      if (++st == kStages) st = 0, ph ^= 1;

      // ---- the item's end, or the run's: the warps' sums together
      const bool ends_here = p.tile + 1 == p.tiles;
      if (ends_here || f + 1 == f1) {
        const bool begun_here = f - p.tile >= f0;
        // (scales in registers of their own: with the loop's, 8 sequences of up to 131072
        // tokens take 111.3 us, so 109.2)
        float m[NB][2], l[NB][2], qj[NB][2];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            asm volatile("mov.b32 %0, %1;" : "=f"(qj[nb][c]) : "f"(qs[nb][c]));
            m[nb][c] = mx[nb][c];
            l[nb][c] = sum[nb][c];
            l[nb][c] += __shfl_xor_sync(0xFFFFFFFFu, l[nb][c], 4);
            l[nb][c] += __shfl_xor_sync(0xFFFFFFFFu, l[nb][c], 8);
            l[nb][c] += __shfl_xor_sync(0xFFFFFFFFu, l[nb][c], 16);
          }
        float *part = a.part + (2 * static_cast<int64_t>(me) + begun_here) * S::kPart;
        const bool alone = begun_here && ends_here;  // no other group has a part of it
        together(m, l, qj, [&](int nb, int j, const float4 &v, const float (&ma)[2], const float (&la)[2]) {
          if (alone) {
            finish(p.b, head, row0, nb, j, v, ma, la, qj);
          } else {
            reinterpret_cast<float4 *>(part)[(j * NB + nb) * 32 + lane] = v;
            if (j == 0 && g == 0) {
              *reinterpret_cast<float4 *>(part + kRows * D + (nb * 8 + 2 * t) * 2) =
                  make_float4(ma[0], la[0], ma[1], la[1]);
              *reinterpret_cast<float2 *>(part + kRows * (D + 2) + nb * 8 + 2 * t) =
                  make_float2(qj[nb][0], qj[nb][1]);
            }
          }
        });
        if (!alone) {
          meet();
          if (tid == 0)  // (the addition releases what the barrier has gathered)
            bars.ticket[begun_here] = atom_add_acq_rel_gpu(a.tickets + p.b * plan.items + p.item, 1u);
          if (begun_here) late = p, has_late = true;
          else early = p, has_early = true;
        }
      }
    }
    // ---- items that other groups have parts of: the last to leave its part sums all of
    // them, every warp each fourth one in the order of the tokens (a warp's quarter of all
    // of them, four in flight: 57 parts took 9 to 14 us)
    if (has_early || has_late) {
      meet();
#pragma unroll 1
      for (int n = 0; n < 2; ++n) {
        if (!(n ? has_late : has_early)) continue;
        const Place &e = n ? late : early;
        const int s0 = first[e.b] * plan.items + e.item * (e.tiles + kJoinSlots);
        const int c0 = plan.group_of(s0), c1 = plan.group_of(s0 + e.tiles - 1);
        if (bars.ticket[n] != static_cast<uint32_t>(c1 - c0)) continue;
        if (tid == 0) a.tickets[e.b * plan.items + e.item] = 0u;
        __threadfence();
        const int hd = e.item / blocks, r0 = (e.item - hd * blocks) * kRows;
        float m[NB][2], l[NB][2], qb[NB][2];
        const float *part0 = a.part + (2 * static_cast<int64_t>(c0) + 1) * S::kPart;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          const float2 by2 = __ldcg(reinterpret_cast<const float2 *>(part0 + kRows * (D + 2) + nb * 8 + 2 * t));
          qb[nb][0] = by2.x, qb[nb][1] = by2.y;
          m[nb][0] = m[nb][1] = -INFINITY, l[nb][0] = l[nb][1] = 0.0f;
#pragma unroll
          for (int j = 0; j < kTiles; ++j)
#pragma unroll
            for (int c = 0; c < 4; ++c) o[j][nb][c] = 0.0f;
        }
        for (int c = c0 + warp; c <= c1; c += kWarps) {
          // the item begins in the second part of its first group, and goes on in the
          // first one of each of the others
          const float *part = a.part + (2 * static_cast<int64_t>(c) + (c == c0)) * S::kPart;
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            const float4 st4 = __ldcg(reinterpret_cast<const float4 *>(part + kRows * D + (nb * 8 + 2 * t) * 2));
            float4 x[kTiles];
#pragma unroll
            for (int j = 0; j < kTiles; ++j)
              x[j] = __ldcg(reinterpret_cast<const float4 *>(part) + (j * NB + nb) * 32 + lane);
            const float u0 = fmaxf(m[nb][0], st4.x), u1 = fmaxf(m[nb][1], st4.z);
            const float a0 = factor(m[nb][0], u0, qb[nb][0]), a1 = factor(m[nb][1], u1, qb[nb][1]);
            const float b0 = factor(st4.x, u0, qb[nb][0]), b1 = factor(st4.z, u1, qb[nb][1]);
            m[nb][0] = u0, m[nb][1] = u1;
            l[nb][0] = l[nb][0] * a0 + st4.y * b0, l[nb][1] = l[nb][1] * a1 + st4.w * b1;
#pragma unroll
            for (int j = 0; j < kTiles; ++j) {
              o[j][nb][0] = o[j][nb][0] * a0 + x[j].x * b0, o[j][nb][1] = o[j][nb][1] * a1 + x[j].y * b1;
              o[j][nb][2] = o[j][nb][2] * a0 + x[j].z * b0, o[j][nb][3] = o[j][nb][3] * a1 + x[j].w * b1;
            }
          }
        }
        together(m, l, qb, [&](int nb, int j, const float4 &v, const float (&ma)[2], const float (&la)[2]) {
          finish(e.b, hd, r0, nb, j, v, ma, la, qb);
        });
      }
    }
    // ---- sequences without a cached token: zeros
    const int64_t rows = static_cast<int64_t>(a.Tq) * a.HK * a.G;
    for (int b = me; b < a.B; b += everyone) {
      if (first[b + 1] != first[b]) continue;
      for (int64_t e = tid; e < rows * (D / 4); e += kWarps * 32) {
        const int64_t row = e / (D / 4), i = row / (a.HK * a.G), h = row - i * (a.HK * a.G);
        *reinterpret_cast<uint2 *>(a.y + (static_cast<int64_t>(b) * a.Tq + i) * a.y_ts + h * a.y_hs +
                                   e % (D / 4) * 4) = make_uint2(0, 0);
      }
    }
  }
  __syncthreads();
  if (threadIdx.x < kGroups && *static_cast<volatile uint32_t *>(&all_bars[threadIdx.x].abort))
    atomicMax(a.status, kStatusTimeout);
}

// ---------------------------------------------------------------- the weights

// weights[page][head][place] += sum over the query rows of exp2((s - max) * scale) / sum,
// from the products that the attention left: a thread has one cached token.  A thread is
// the only one to add to its place, unless sequences share a page.
constexpr int kWeightThreads = 256;
static_assert(kLift == 7.0f, "the weights are divided by sums of 2^7 p");
__global__ void __launch_bounds__(kWeightThreads) kv4_weights_kernel(const Kv4AttnArgs a) {
  __shared__ float2 stat[kKv4MaxRows];
  __shared__ float inv[kKv4MaxRows];
  griddep_launch_dependents();
  griddep_wait();
  const int R = a.G * a.Tq, h = blockIdx.y % a.HK, b = blockIdx.y / a.HK;
  const int len = min(max(__ldg(a.lens + b), 0), a.max_len);
  if (blockIdx.x * kWeightThreads >= len) return;
  const int64_t bh = static_cast<int64_t>(b) * a.HK + h;
  for (int r = threadIdx.x; r < R; r += kWeightThreads) {
    const float4 row = *reinterpret_cast<const float4 *>(a.stats + (bh * R + r) * 4);
    stat[r] = make_float2(row.x, row.y);
    // (the sum's p are 2^kLift times as large; a row that sees nothing adds nothing)
    inv[r] = row.z == 0.0f ? 0.0f : 128.0f / row.z;
  }
  __syncthreads();
  const int tok = blockIdx.x * kWeightThreads + threadIdx.x;
  if (tok >= len) return;
  const int page = __ldg(a.table + static_cast<int64_t>(b) * a.width + (tok >> a.page_log2));
  if (page < 0 || page >= a.pages) return;
  const float *s = a.logits + bh * R * a.max_len + tok;
  float w = 0.0f;
  for (int r = 0; r < R; ++r) {
    const float v = s[static_cast<int64_t>(r) * a.max_len];
    if (v != -INFINITY) w += ex2((v - stat[r].x) * stat[r].y) * inv[r];
  }
  atomicAdd(a.weights + ((static_cast<int64_t>(page) * a.HK + h) << a.page_log2) + (tok & ((1 << a.page_log2) - 1)), w);
}

// ---------------------------------------------------------------- host

constexpr int kMaxSms = 160;  // more than a GB300 has

struct Layout {
  size_t tickets, part, stats, logits, total;
};
Layout layout(int64_t B, int64_t Tq, int64_t HQ, int64_t HK, int64_t D, int64_t max_len, bool weights) {
  auto up = [](size_t v) { return (v + 255) / 256 * 256; };
  Layout l;
  // the tickets' place and size are the same for all sizes, so that one workspace
  // serves calls of several
  l.tickets = 256;
  l.part = l.tickets + kKv4MaxItems * 4;
  l.stats = l.part + up(static_cast<size_t>(2) * 3 * kMaxSms * 16 * (D + 3) * 4);
  const size_t rows = static_cast<size_t>(B) * HQ * Tq;
  l.logits = l.stats + (weights ? up(rows * 16) : 0);
  l.total = l.logits + (weights ? up(rows * static_cast<size_t>(max_len) * 4) : 0);
  return l;
}

}  // namespace

size_t kv4_workspace(int64_t B, int64_t Tq, int64_t HQ, int64_t HK, int64_t D, int64_t max_len,
                     bool weights) {
  return layout(B, Tq, HQ, HK, D, max_len, weights).total;
}

cudaError_t launch_kv4_attention(Kv4AttnArgs a, void *ws, int num_sms, cudaStream_t st) {
  const Layout l = layout(a.B, a.Tq, static_cast<int64_t>(a.HK) * a.G, a.HK, a.D, a.max_len, a.weights != nullptr);
  uint8_t *at = static_cast<uint8_t *>(ws);
  a.status = static_cast<uint32_t *>(ws);
  a.tickets = reinterpret_cast<uint32_t *>(at + l.tickets);
  a.part = reinterpret_cast<float *>(at + l.part);
  if (a.weights) {
    a.stats = reinterpret_cast<float *>(at + l.stats);
    a.logits = reinterpret_cast<float *>(at + l.logits);
  }
  const int R = a.G * a.Tq;
  auto run = [&](auto d, auto n) {
    constexpr int D = decltype(d)::value, NB = decltype(n)::value;
    using S = Sizes<D, NB>;
    cudaError_t e = allow_smem<kv4_attention_kernel<D, NB>>(S::kSmem + (kKv4MaxBatch + 1) * 4);
    if (e != cudaSuccess) return e;
    // setmaxnreg.inc waits for registers that the block was launched with: no launch
    // unless the compiled count covers the split
    static const int regs = [] {
      cudaFuncAttributes fa;
      return cudaFuncGetAttributes(&fa, kv4_attention_kernel<D, NB>) == cudaSuccess ? fa.numRegs : 0;
    }();
    if (S::kGroups > 1 && regs * S::kThreads < 128 * (S::kGroups * S::kRegs + S::kCopyRegs))
      return cudaErrorInvalidConfiguration;
    const int64_t tiles = static_cast<int64_t>(a.B) * a.HK * ((R + S::kRows - 1) / S::kRows) *
                          ((a.max_len + S::kTile - 1) / S::kTile);
    const int64_t grid = tiles < num_sms ? (tiles < 1 ? 1 : tiles) : num_sms;
    return launch_pdl(kv4_attention_kernel<D, NB>,
                      dim3(static_cast<unsigned>(grid < kMaxSms ? grid : kMaxSms)), dim3(S::kThreads),
                      S::kSmem + (a.B + 1) * 4, st, a);
  };
  auto by_rows = [&](auto d) {
    return R <= 8 ? run(d, std::integral_constant<int, 1>{}) : run(d, std::integral_constant<int, 2>{});
  };
  cudaError_t e = a.D == 64    ? by_rows(std::integral_constant<int, 64>{})
                  : a.D == 128 ? by_rows(std::integral_constant<int, 128>{})
                               : by_rows(std::integral_constant<int, 256>{});
  if (e != cudaSuccess || !a.weights || a.max_len == 0) return e;
  return launch_pdl(kv4_weights_kernel,
                    dim3((a.max_len + kWeightThreads - 1) / kWeightThreads, a.B * a.HK),
                    dim3(kWeightThreads), 0, st, a);
}

}  // namespace fp8bq
