// prompt_attention.cu -- causal attention over whole prompts: packed sequences of
// different lengths, grouped heads.
//
// Per sequence (rows offsets[s] .. offsets[s+1]-1), token i and head h:
//   s_j = scale * q_i . k_j for j <= i,  y_i = sum_j softmax(s)_j v_j
// in one pass over the keys with the running maximum and sum of the softmax.
//
// Bound by the tensor cores: 4 D operations a pair of query row and key.  A unit of
// work is a key/value head of 2 x 128 query rows: floor(128 / G) tokens x G heads
// each (G = HQ / HK), so that the rows of short sequences fill the tiles, and all
// heads of a group share the keys and values that are read.  Per tile of 128 keys
//   S = Q K^T    both operands in shared memory (TMA, 128-byte swizzle), S in TMEM
//   P = exp2(S - max), BF16, written over S's own columns
//   O += P V     P from TMEM, V as TMA left it (N-major), O in TMEM
// The two row tiles alternate: while the tensor cores work for one, the other's
// four warps (a thread a row) compute its P.  TMEM holds 2 x (128 S + 128 O) columns,
// which is all of it (with heads up to 64, whose O has 64, 128 stay idle).
// O is rescaled only when a row's maximum has grown by more than 2^8 since its last
// reference (p <= 2^8 until then; the row's sum is held to the same reference).
// P is rounded to BF16 (half a step, 2^-8 of a p): kind::f16 takes both operands in
// one type, and V is BF16.
//
// Measured: 16384 tokens, 32 heads over 4 of 128: 1.22 to 1.35 ms, with the power cap (all
// at the cap: 1.63 PFLOP/s of what the causal triangle needs, where cuBLAS has 1.74).  A
// pair of steps takes 2630 cycles, of which the tensor cores' 2150: a tile's chain is 1200
// for its softmax, 150 until its products begin and 1280 until the next scores are there.
// A unit's end costs some 4000 more, and 12 to 19 % of the tensor work of short prompts goes
// to pairs of a unit's last tiles that the mask hides: nine ragged prompts of 4099 tokens
// together, 64 heads over 8, take 72.5 us, 0.48 of cuBLAS's rate.  CTA pairs sharing K and V
// (cta_group::2) gained 2 % and are left out.
#include "common.cuh"
#include "ptx.cuh"

namespace fp8bq {
namespace {

constexpr int kKeys = 128;                 // keys a tile
constexpr int kThreads = 384;              // 2 x 4 softmax warps, 2 MMA warps, copy warp, 1 idle
constexpr int kMmaWarp = 8, kCopyWarp = 10;
// registers: a softmax thread holds a row's 128 scores, which the third warpgroup
// makes room for (384 x 168 at launch)
constexpr int kHighRegs = 224, kLowRegs = 56;
constexpr int kHalf = 128 * 128;           // bytes of 128 rows x 64 values
constexpr float kGrowth = 8.0f;            // log2: a maximum within it keeps its reference

template <int DP>
struct Cfg {
  static constexpr int kHalves = DP / 64;
  static constexpr int kTileBytes = kHalves * kHalf;  // 128 rows of Q, K or V
  static constexpr int kStages = DP == 128 ? 4 : 8;
  static constexpr int kOutBytes = 8 * 32 * 64;       // a softmax warp's 32 rows x 32 values
  static constexpr int kSmem = (2 + kStages) * kTileBytes + kOutBytes + 1024;  // 1024: alignment
};

struct Unit {
  int start;   // the sequence's first row
  int len;     // its tokens
  int t0;      // the unit's first token
  int head;    // key/value head
  int tiles;   // key tiles; 0: no more units
};

struct Shared {
  uint64_t q_full[2], q_empty[2];
  uint64_t kv_full[8], kv_empty[8];
  uint64_t s_full[2], p_ready[2], o_done[2], o_free[2];
  uint64_t v_clean[2], u_full[2], u_empty[2], turn[2], done[2];
  uint32_t abort, tmem;
  Unit unit[2];
  // Tokens of the last tiles with a value that is not finite, a bit each.  Those tiles are
  // two at most: a unit of one head a group has 256 tokens from a multiple of 256 on, one
  // of more heads no more than 128.
  alignas(16) uint32_t bad[2][8];
  int bound[kMaxPrompts + 1];
  int blocks[kMaxPrompts];
};

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float reciprocal(float x) {  // within 2^-23
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Units in the order of their work, the longest first: block l of every sequence
// that has more than l blocks, for l from the top; a block's key/value heads are
// neighbours.  Runs on one warp.
struct Units {
  const int *blocks;
  int S, top, HK;
  int64_t total;
  __device__ int64_t above(int level, int lane) const {  // blocks at `level` and above
    int n = 0;
    for (int s = lane; s < S; s += 32) n += max(blocks[s] - level, 0);
    return __reduce_add_sync(0xFFFFFFFFu, n);
  }
  __device__ void find(int64_t u, int lane, int &seq, int &block, int &head) const {
    const int rank = static_cast<int>(u / HK);
    head = static_cast<int>(u - static_cast<int64_t>(rank) * HK);
    int lo = 0, hi = top;  // the last level with above(level) > rank
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (above(mid, lane) > rank) lo = mid; else hi = mid;
    }
    block = lo;
    int k = rank - static_cast<int>(above(lo + 1, lane));  // the k-th sequence with that block
    seq = 0;
    for (int s0 = 0; s0 < S; s0 += 32) {
      uint32_t has = __ballot_sync(0xFFFFFFFFu, s0 + lane < S && blocks[s0 + lane] > lo);
      const int n = __popc(has);
      if (k < n) {
        for (; k > 0; --k) has &= has - 1;
        seq = s0 + __ffs(has) - 1;
        break;
      }
      k -= n;
    }
  }
};

// DP: the head size that tiles are laid out for, FULL: a.D is that, so that S has as many
// steps (asked at each step: 2 % of 16384 tokens)
template <int DP, bool FULL>
__global__ void __launch_bounds__(kThreads, 1)
prompt_attention_kernel(const __grid_constant__ CUtensorMap qm, const __grid_constant__ CUtensorMap km,
                        const __grid_constant__ CUtensorMap vm, const PromptArgs a) {
  using C = Cfg<DP>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = smem_raw + (1024 - (smem_u32(smem_raw) & 1023)) % 1024;
  uint8_t *ring = smem + 2 * C::kTileBytes;
  __shared__ Shared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  volatile uint32_t *abort = &sh.abort;
  const uint64_t limit = a.wait_limit_ns;
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.q_full[i], 1);
      mbar_init(&sh.s_full[i], 1), mbar_init(&sh.o_done[i], 1);
      mbar_init(&sh.p_ready[i], 4), mbar_init(&sh.o_free[i], 4);
      mbar_init(&sh.u_full[i], 1), mbar_init(&sh.u_empty[i], 10);
      mbar_init(&sh.v_clean[i], 8), mbar_init(&sh.q_empty[i], 1);
      mbar_init(&sh.turn[i], 1), mbar_init(&sh.done[i], 1);
    }
    for (int i = 0; i < C::kStages; ++i) mbar_init(&sh.kv_full[i], 1), mbar_init(&sh.kv_empty[i], 2);
    sh.abort = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&sh.tmem, 512);
    tmem_relinquish();
  }
  if (warp == kCopyWarp && lane == 0) tma_prefetch_desc(&qm), tma_prefetch_desc(&km), tma_prefetch_desc(&vm);
  griddep_launch_dependents();
  griddep_wait();
  const int G = a.HQ / a.HK, half_tokens = 128 / G, unit_tokens = 2 * half_tokens;
  for (int s = tid; s <= a.S; s += kThreads) sh.bound[s] = min(max(__ldg(a.offsets + s), 0), a.T);
  __syncthreads();
  for (int s = tid; s < a.S; s += kThreads)
    sh.blocks[s] = (max(sh.bound[s + 1] - sh.bound[s], 0) + unit_tokens - 1) / unit_tokens;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;

  if (warp == kCopyWarp) {
    // ---- copies, and the units for everybody
    setmaxnreg_dec<kLowRegs>();
    Units units = {sh.blocks, a.S, 0, a.HK, 0};
    int top = 0;
    for (int s = lane; s < a.S; s += 32) top = max(top, sh.blocks[s]);
    units.top = __reduce_max_sync(0xFFFFFFFFu, top);
    units.total = units.above(0, lane) * a.HK;
    const int64_t grid = gridDim.x, cta = blockIdx.x;
    const uint32_t q_bytes = C::kHalves * half_tokens * G * 128;
    int64_t c = 0;         // copies into the ring so far
    uint32_t queries = 0;  // and of queries, the row tiles in turn
    bool ok = true;
    int k = 0;
    auto ring_copy = [&](const CUtensorMap *map, int head, int row, bool skip) {
      const int st = static_cast<int>(c % C::kStages);
      if (!mbar_wait(&sh.kv_empty[st], (c / C::kStages & 1) ^ 1, abort, limit)) return false;
      mbar_arrive_expect_tx(&sh.kv_full[st], C::kTileBytes);
      ++c;
      if (skip) return true;
#pragma unroll
      for (int h = 0; h < C::kHalves; ++h)
        tma_load_3d(ring + st * C::kTileBytes + h * kHalf, map, &sh.kv_full[st], h * 64, head, row);
      return true;
    };
    for (;; ++k) {
      // rounds in turn from the left and from the right: equal sums
      const int64_t u = k * grid + (k & 1 ? grid - 1 - cta : cta);
      Unit un = {0, 0, 0, 0, 0};
      if (u < units.total) {
        int seq, block;
        units.find(u, lane, seq, block, un.head);
        un.start = sh.bound[seq];
        un.len = sh.bound[seq + 1] - un.start;
        un.t0 = block * unit_tokens;
        un.tiles = (min(un.len, un.t0 + unit_tokens) + kKeys - 1) / kKeys;
      }
      if (lane == 0) {
        ok = mbar_wait(&sh.u_empty[k & 1], (k >> 1 & 1) ^ 1, abort, limit);
        if (ok) {
          sh.unit[k & 1] = un;
          for (int w = 0; w < 8; w += 4) *reinterpret_cast<uint4 *>(&sh.bad[k & 1][w]) = make_uint4(0, 0, 0, 0);
          mbar_arrive(&sh.u_full[k & 1]);
        }
        if (ok && un.tiles > 0) {
          ok = ring_copy(&km, un.head, un.start, a.fault && cta == 0 && k == 0);
          for (int i = 0; i < 2 && ok; ++i) {
            ok = mbar_wait(&sh.q_empty[i], (k & 1) ^ 1, abort, limit);
            if (!ok) break;
            mbar_arrive_expect_tx(&sh.q_full[i], q_bytes);
            ++queries;
#pragma unroll
            for (int h = 0; h < C::kHalves; ++h)
              tma_load_3d(smem + i * C::kTileBytes + h * kHalf, &qm, &sh.q_full[i], h * 64,
                          un.head * G, un.start + un.t0 + i * half_tokens);
          }
          ok = ok && ring_copy(&vm, un.head, un.start, false);
          for (int j = 1; j < un.tiles && ok; ++j)
            ok = ring_copy(&km, un.head, un.start + j * kKeys, false) &&
                 ring_copy(&vm, un.head, un.start + j * kKeys, false);
        }
      }
      ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
      if (!ok || un.tiles == 0) break;
    }
    if (lane == 0) {
      // Copies in flight land before the memory is given up, also those that nobody waits
      // for any more: another role may give up at any time, after the last copy too.
      for (int64_t i = c < C::kStages ? 0 : c - C::kStages; i < c; ++i)
        mbar_wait_alone(&sh.kv_full[i % C::kStages], i / C::kStages & 1, limit);
#pragma unroll
      for (uint32_t i = 0; i < 2; ++i)
        if (queries > i) mbar_wait_alone(&sh.q_full[i], (queries - 1 - i) >> 1 & 1, limit);
    }
    __syncwarp();
  } else if (warp == kMmaWarp || warp == kMmaWarp + 1) {
    // ---- products of row tile i: S first, then P V and the next S as one block.  The
    // whole warp walks; one lane of it issues a block and its commits in one branch
    // (each by itself under a lane's predicate: 90 cycles an MMA, which takes the tensor
    // cores 67; 16384 tokens, 32 heads over 4: 1520 us, so 1450).  A commit takes 97
    // cycles.  So each tile has an issuer of its own, and they pass the turn: while one
    // commits and waits, the other's MMAs run.  (Without turns both tiles' blocks
    // mingle, both S come late and nothing runs beside the softmax: 1950 us; one issuer
    // for both: 1620.)  P is waited for last, with the turn in hand: once it is there
    // nothing but the issue is left (before the turn: 1397 against 1343 us, on one GPU).
    setmaxnreg_dec<kLowRegs>();
    const int i = warp - kMmaWarp;
    const uint32_t s_desc = idesc_bf16(128, kKeys), o_desc = idesc_bf16(128, a.D, true);
    const uint64_t q_at = sdesc_kmajor_sw128(smem_u32(smem)) + i * (C::kTileBytes / 16);
    const uint64_t k_base = sdesc_kmajor_sw128(smem_u32(ring));
    const uint64_t v_base = sdesc_nmajor_sw128(smem_u32(ring), kHalf);
    const uint32_t s_at = tmem + i * 128, o_at = tmem + 256 + i * 128;
    const int steps = a.D / 16;
    uint32_t pph = 0, tph = i ^ 1, looked = 0;  // tiles whose values were looked through
    int st = 0;
    uint32_t ring_ph = 0;  // the ring's place and round
    bool ok = true;
    auto wait = [&](uint64_t *bar, uint32_t parity) {
      return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, abort, limit));
    };
    auto scores = [&](int at) {
      const uint64_t kd = k_base + at * (C::kTileBytes / 16);
#pragma unroll
      for (int s = 0; s < DP / 16; ++s) {
        const uint64_t off = (s >> 2) * (kHalf / 16) + (s & 3) * 2;
        if (FULL || s < steps) umma_bf16(s_at, q_at + off, kd + off, s_desc, s > 0);
      }
    };
    for (int k = 0; ok; ++k) {
      ok = wait(&sh.u_full[k & 1], k >> 1 & 1);
      if (!ok) break;
      const int tiles = __shfl_sync(0xFFFFFFFFu, sh.unit[k & 1].tiles, 0);
      const int special = __shfl_sync(0xFFFFFFFFu, sh.unit[k & 1].t0, 0) / kKeys;
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.u_empty[k & 1]);
      if (tiles == 0) break;
      ok = wait(&sh.kv_full[st], ring_ph) && wait(&sh.q_full[i], k & 1) && wait(&sh.turn[i], tph);
      tph ^= 1;
      if (!ok) break;
      tc_fence_after();
      if (elect_one()) {
        scores(st);
        mbar_arrive(&sh.turn[i ^ 1]);
        umma_commit(&sh.s_full[i]);
        umma_commit(&sh.kv_empty[st]);
        if (tiles == 1) umma_commit(&sh.q_empty[i]);
      }
      __syncwarp();
      if (++st == C::kStages) st = 0, ring_ph ^= 1;
      for (int j = 0; j < tiles; ++j) {
        const int vs = st;
        const bool more = j + 1 < tiles;
        ok = wait(&sh.kv_full[vs], ring_ph);
        if (++st == C::kStages) st = 0, ring_ph ^= 1;
        if (ok && more) ok = wait(&sh.kv_full[st], ring_ph);
        if (ok && j >= special) {
          ok = wait(&sh.v_clean[looked & 1], looked >> 1 & 1);
          ++looked;
        }
        if (ok && j == 0) ok = wait(&sh.o_free[i], (k & 1) ^ 1);
        ok = ok && wait(&sh.turn[i], tph) && wait(&sh.p_ready[i], pph);
        tph ^= 1, pph ^= 1;
        if (!ok) break;
        tc_fence_after();
        const uint64_t vd = v_base + vs * (C::kTileBytes / 16);
        if (elect_one()) {
#pragma unroll
          for (int s = 0; s < kKeys / 16; ++s)
            umma_bf16_ta(o_at, s_at + s * 8, vd + s * (2048 / 16), o_desc, j > 0 || s > 0);
          if (more) scores(st);
          mbar_arrive(&sh.turn[i ^ 1]);
          if (more) umma_commit(&sh.s_full[i]);
          umma_commit(&sh.o_done[i]);
          umma_commit(&sh.kv_empty[vs]);
          if (more) umma_commit(&sh.kv_empty[st]);
          if (j + 2 == tiles) umma_commit(&sh.q_empty[i]);
        }
        __syncwarp();
        if (more && ++st == C::kStages) st = 0, ring_ph ^= 1;
      }
    }
    if (elect_one()) {
      umma_commit(&sh.done[i]);
      mbar_wait_alone(&sh.done[i], 0, limit);
    }
    __syncwarp();
  } else if (warp < 8) {
    // ---- softmax: a thread a row of tile i
    setmaxnreg_inc<kHighRegs>();
    const int i = warp >> 2, row = tid & 127;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_at = tmem + lanes + i * 128, o_at = tmem + lanes + 256 + i * 128;
    const int tok_in = row / G, head_in = row - tok_in * G;
    const float sc = a.scale_log2;
    uint4 *out = reinterpret_cast<uint4 *>(ring + C::kStages * C::kTileBytes) + warp * 128;
    uint32_t sph = 0, oph = 0, looked = 0;
    int64_t c = 0;  // copies into the ring of the units before
    bool ok = true;
    for (int k = 0;; ++k) {
      ok = __all_sync(0xFFFFFFFFu, mbar_wait(&sh.u_full[k & 1], k >> 1 & 1, abort, limit));
      if (!ok) break;
      Unit un = sh.unit[k & 1];
      if (un.tiles == 0) break;
      const int tok = un.t0 + i * half_tokens + tok_in;
      const int special = un.t0 / kKeys;
      float ref = -INFINITY, sum = 0.0f;
      for (int j = 0; j < un.tiles && ok; ++j) {
        if (j >= special) {
          // values of these tokens are hidden from some rows: one that is not finite would
          // spoil those (0 times it is NaN), so it is taken out here and added to the rows
          // that see it at the end.  (One warp for it, beside the others, took 3800 cycles
          // that the last product waited for.)
          const int64_t n = c + 2 * j + 1;
          ok = __all_sync(0xFFFFFFFFu, mbar_wait(&sh.kv_full[n % C::kStages], n / C::kStages & 1, abort, limit));
          if (!ok) break;
          uint4 *v = reinterpret_cast<uint4 *>(ring + (n % C::kStages) * C::kTileBytes) + tid;
          // halves whose exponent is all ones
          auto flags = [](uint32_t y) { return ((y & 0x7F807F80u) + 0x00800080u) & 0x80008000u; };
          auto clean = [&](uint32_t y) {
            const uint32_t f = flags(y);
            return y & ~((f >> 31) * 0xFFFF0000u) & ~((f >> 15 & 1u) * 0xFFFFu);
          };
          constexpr int kWords = C::kTileBytes / 16 / 256;
          uint4 x[kWords];
          uint32_t f = 0;
#pragma unroll
          for (int w = 0; w < kWords; ++w) x[w] = v[w * 256];
#pragma unroll
          for (int w = 0; w < kWords; ++w) f |= flags(x[w].x) | flags(x[w].y) | flags(x[w].z) | flags(x[w].w);
          if (f) {
#pragma unroll
            for (int w = 0; w < kWords; ++w) {
              if (!(flags(x[w].x) | flags(x[w].y) | flags(x[w].z) | flags(x[w].w))) continue;
              v[w * 256] = make_uint4(clean(x[w].x), clean(x[w].y), clean(x[w].z), clean(x[w].w));
              // (8 words of 16 bytes a token and half)
              atomicOr(&sh.bad[k & 1][(j - special) * 4 + (w & 3)], 1u << (tid >> 3));
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          // (two barriers in turn: one tile's four warps may be a tile ahead)
          if (lane == 0) mbar_arrive(&sh.v_clean[looked & 1]);
          ++looked;
        }
        ok = __all_sync(0xFFFFFFFFu, mbar_wait(&sh.s_full[i], sph, abort, limit));
        sph ^= 1;
        if (!ok) break;
        tc_fence_after();
        uint32_t s[128];
#pragma unroll
        for (int q = 0; q < 4; ++q) tmem_ld32(s_at + q * 32, s + q * 32);
        tmem_ld_wait();
        const int seen = tok - j * kKeys + 1;  // keys of the tile that the row sees
        if (__any_sync(0xFFFFFFFFu, seen < kKeys)) {
#pragma unroll
          for (int x = 0; x < 128; ++x)
            if (x >= seen) s[x] = 0xFF800000u;  // -inf
        }
        float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int x = 0; x < 128; x += 2)
          m[x >> 1 & 3] = max3(m[x >> 1 & 3], __uint_as_float(s[x]), __uint_as_float(s[x + 1]));
        const float top = fmaxf(max3(m[0], m[1], m[2]), m[3]);
        const bool grow = (top - ref) * sc > kGrowth;
        if (j == 0) {
          ref = top;
        } else if (__any_sync(0xFFFFFFFFu, grow)) {
          const float by = grow ? ex2((ref - top) * sc) : 1.0f;
          if (grow) ref = top;
          sum *= by;
          ok = __all_sync(0xFFFFFFFFu, mbar_wait(&sh.o_done[i], oph ^ 1, abort, limit));
          if (!ok) break;
          tc_fence_after();
#pragma unroll 1
          for (int q = 0; q < DP / 32; ++q) {
            uint32_t o[32];
            tmem_ld32(o_at + q * 32, o);
            tmem_ld_wait();
#pragma unroll
            for (int x = 0; x < 32; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * by);
            tmem_st32(o_at + q * 32, o);
          }
        }
        oph ^= 1;
        // (the difference is taken before the scale, so that it is exact where it is
        // small, however large the scores are; one rounding less, s * sc - ref * sc, is
        // 2 % faster and gives infinite p where ref * sc passes 2^30)
        const float neg = ref == -INFINITY ? 0.0f : -ref;
        const uint64_t sc2 = pair(sc, sc), neg2 = pair(neg, neg);
        uint64_t l[2] = {0, 0};
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          uint32_t p[32];
#pragma unroll
          for (int x = 0; x < 32; ++x) {
            float p0, p1;
            unpair(mul2(add2(pair(__uint_as_float(s[q * 64 + 2 * x]), __uint_as_float(s[q * 64 + 2 * x + 1])),
                             neg2), sc2), p0, p1);
            p0 = ex2(p0), p1 = ex2(p1);
            l[x & 1] = add2(l[x & 1], pair(p0, p1));
            p[x] = pack_bf16(p0, p1);
          }
          tmem_st32(s_at + q * 32, p);
        }
        float l0, l1;
        unpair(add2(l[0], l[1]), l0, l1);
        sum += l0 + l1;
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.p_ready[i]);
      }
      if (!ok) break;
      c += 2 * un.tiles;
      // ---- the unit's end
      ok = __all_sync(0xFFFFFFFFu, mbar_wait(&sh.o_done[i], oph ^ 1, abort, limit));
      if (!ok) break;
      tc_fence_after();
      const volatile uint32_t *bad_tokens = sh.bad[k & 1];
      const bool bad = __any_sync(0xFFFFFFFFu, bad_tokens[lane & 7] != 0);
      const bool live = tok_in < half_tokens && tok < un.len;
      const float by = reciprocal(sum);
      const int64_t y_at = live ? static_cast<int64_t>(un.start + tok) * a.y_ts +
                                      static_cast<int64_t>(un.head * G + head_in) * a.y_hs
                                : -1;
      // by way of shared memory, so that four lanes write 64 bytes of a row (a row a
      // lane: 16 bytes of 32 rows a store).  Little code: what runs once a unit comes
      // from afar.
      const int piece = lane & 3;
      int64_t to[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) to[x] = __shfl_sync(0xFFFFFFFFu, y_at, x * 8 + (lane >> 2));
#pragma unroll 1
      for (int q = 0; q < DP / 32; ++q) {
        uint32_t o[32];
        tmem_ld32(o_at + q * 32, o);
        tmem_ld_wait();
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          uint32_t w[4];
#pragma unroll
          for (int z = 0; z < 4; ++z)
            w[z] = pack_bf16(__uint_as_float(o[x * 8 + 2 * z]) * by, __uint_as_float(o[x * 8 + 2 * z + 1]) * by);
          out[lane * 4 + (x ^ (lane >> 1 & 3))] = make_uint4(w[0], w[1], w[2], w[3]);
        }
        __syncwarp();
        uint4 v[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int r = x * 8 + (lane >> 2);
          v[x] = out[r * 4 + (piece ^ (r >> 1 & 3))];
        }
        const bool in = q * 32 + piece * 8 < a.D;
#pragma unroll
        for (int x = 0; x < 4; ++x)
          if (in && to[x] >= 0) *reinterpret_cast<uint4 *>(a.y + to[x] + q * 32 + piece * 8) = v[x];
        __syncwarp();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.o_free[i]);
      if (bad && live) {
        // what was taken out of the tokens that the row sees, eight values at a time (the
        // row is written; an infinity or a NaN outdoes its rounding).  Marked tokens alone:
        // with all of them, value by value, one NaN in 4096 tokens made 94 us 1770.
        const int last = tok - special * kKeys;
        const uint16_t *v = a.v + static_cast<int64_t>(un.start + special * kKeys) * a.v_ts +
                            static_cast<int64_t>(un.head) * a.v_hs;
#pragma unroll 1
        for (int x = 0; x < a.D; x += 8) {
          float e[8] = {-0.0f, -0.0f, -0.0f, -0.0f, -0.0f, -0.0f, -0.0f, -0.0f};  // (x + -0 is x)
          bool any = false, full = false;  // full: nothing but NaN
#pragma unroll 1
          for (int w = 0; w * 32 <= last && !full; ++w) {
            uint32_t left = bad_tokens[w];
            if (last - w * 32 < 31) left &= (2u << (last - w * 32)) - 1u;
#pragma unroll 1
            for (; left && !full; left &= left - 1u) {
              const int t = w * 32 + __ffs(left) - 1;
              const uint4 r = __ldg(reinterpret_cast<const uint4 *>(v + t * a.v_ts + x));
              const uint32_t words[4] = {r.x, r.y, r.z, r.w};
              full = true;
#pragma unroll
              for (int z = 0; z < 8; ++z) {
                const uint32_t b = z & 1 ? words[z >> 1] & 0xFFFF0000u : words[z >> 1] << 16;
                if ((b & 0x7F800000u) == 0x7F800000u) e[z] += __uint_as_float(b), any = true;
                full = full && e[z] != e[z];
              }
            }
          }
          if (!any) continue;
          uint4 *y = reinterpret_cast<uint4 *>(a.y + y_at + x);
          const uint4 r = __ldcg(y);
          const uint32_t words[4] = {r.x, r.y, r.z, r.w};
          uint32_t o[4];
#pragma unroll
          for (int z = 0; z < 4; ++z)
            o[z] = pack_bf16(__uint_as_float(words[z] << 16) + e[2 * z],
                             __uint_as_float(words[z] & 0xFFFF0000u) + e[2 * z + 1]);
          *y = make_uint4(o[0], o[1], o[2], o[3]);
        }
      }
      __syncwarp();  // (every lane is done with the marks)
      if (lane == 0) mbar_arrive(&sh.u_empty[k & 1]);
    }
  } else {
    setmaxnreg_dec<kLowRegs>();
  }
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && *abort) atomicMax(a.status, kStatusTimeout);
  if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

}  // namespace

cudaError_t launch_prompt_attention(const PromptArgs &a, int num_sms, cudaStream_t st) {
  const int G = a.HQ / a.HK, half_tokens = 128 / G;
  CUtensorMap qm, km, vm;
  if (!make_heads_map(&qm, a.q, a.T, a.HQ, a.D, a.q_ts, a.q_hs, half_tokens, G) ||
      !make_heads_map(&km, a.k, a.T, a.HK, a.D, a.k_ts, a.k_hs, kKeys, 1) ||
      !make_heads_map(&vm, a.v, a.T, a.HK, a.D, a.v_ts, a.v_hs, kKeys, 1))
    return cudaErrorInvalidValue;
  // units at most: every sequence may end inside one
  const int64_t blocks = (a.T + 2 * half_tokens - 1) / (2 * half_tokens) + a.S;
  const int64_t most = blocks * a.HK;
  const unsigned grid = static_cast<unsigned>(most < num_sms ? most : num_sms);
  auto run = [&](auto d, auto full) {
    constexpr int DP = decltype(d)::value;
    constexpr bool FULL = decltype(full)::value;
    cudaError_t e = allow_smem<prompt_attention_kernel<DP, FULL>>(Cfg<DP>::kSmem);
    if (e != cudaSuccess) return e;
    // setmaxnreg.inc waits for registers that the block was launched with: no launch
    // unless the compiled count covers the split
    static const int regs = [] {
      cudaFuncAttributes fa;
      return cudaFuncGetAttributes(&fa, prompt_attention_kernel<DP, FULL>) == cudaSuccess ? fa.numRegs : 0;
    }();
    if (regs * kThreads < 256 * kHighRegs + 128 * kLowRegs) return cudaErrorInvalidConfiguration;
    return launch_pdl(prompt_attention_kernel<DP, FULL>, dim3(grid), dim3(kThreads), Cfg<DP>::kSmem, st, qm,
                      km, vm, a);
  };
  auto by_fit = [&](auto d) { return a.D == decltype(d)::value ? run(d, std::true_type{}) : run(d, std::false_type{}); };
  return a.D <= 64 ? by_fit(std::integral_constant<int, 64>{}) : by_fit(std::integral_constant<int, 128>{});
}

}  // namespace fp8bq
