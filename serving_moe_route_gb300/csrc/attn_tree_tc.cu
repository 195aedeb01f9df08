// attn_tree_tc.cu -- moe_attn_tree on the 5th-generation tensor cores, for bf16
// and e4m3 caches.
//
// S = Q K^T and O += P V with tcgen05.mma, 128 rows of (node, query head) by tiles
// of 64 tokens.  A CTA has half of an SM (all of it above head_dim 128): two logit
// tiles S and the accumulator O in tensor memory, Q and a ring of key and value
// tiles in shared memory, and these warps:
//   loads    one warp fills the ring by TMA, as far ahead as it reaches, across
//            unit borders (by cp.async for pages that 8 does not divide), in the
//            order in which tiles are used: K0 K1 V0 K2 V1 ...
//   ready    two warps see to what has landed: e4m3 codes lie in the half of their
//            tile that the same warp will write, and are widened to f16, which
//            holds them exactly.
//   products one thread issues S of the next tile before it waits for the weights
//            of this one.
//   softmax  a warpgroup, a row a thread, one pass with a reference m and the sum
//            l of a row in fp32 (base 2); O is rescaled only when a logit lies LAG
//            above the one that m was taken from.  P is rounded to bf16 (f16 for
//            e4m3 caches) into the columns of S that it has been read from; l adds
//            the weights before that.  bf16 weights leave outputs 1.1 to 1.4 times
//            as far off as their own rounding does; pairs of bf16 mend that and cost
//            2 to 29% (127 us become 164 for the long request below).  f16 weights
//            are lifted to 2^LIFT, which keeps 11 bits down to 2^-27 of the largest.
//   masks    Only tiles that some row does not wholly attend look at masks.  Their
//            weights are 0, but 0 times a value that is not finite is not: such
//            values are replaced by 0 in the tile, and added to O for the rows
//            that do attend them.
// Two CTAs an SM, so that one's products and softmax run under the other's unit
// ends: Q's loads, the last tile's chain of steps and the output take 7 us.
//
// Bound by the softmax's chain in long units: a warp takes 1340 cycles for a tile of
// 64 tokens (reading S 260, maximum 360, weights 530, storing them the rest) and then
// waits 260 for the next S, two CTAs at a time; their products take 1024 for the two,
// shared memory 1500 (a tile moves 96 KB: S 48, O 16, its own arrival 32).  By the
// units' ends in short ones, and by latency in small calls.  Measured on a GB300, 32
// query heads on 4 of 128, bf16: one request of 61 nodes at 131089 tokens 128 us, 1020
// TFLOP/s (53% of cuBLAS's rate); 64 requests of 64 nodes up to 8192: 209 to 219 us,
// 800 to 830 TFLOP/s; of up to 16 nodes, up to 4096: 55 us, 3.2 TB/s; one of 8 nodes
// at 700: 16 us.  e4m3, 128 requests of 8 nodes up to 8192: 135 us, 2.5 TB/s: there a
// tile takes the softmax 2030 beside the warps that widen.
//
// Tried: one CTA an SM with two blocks of rows in turn (the unit ends uncovered: 85 us
// for the batch of 16 nodes); four warps of cp.async instead of TMA, and the fence
// between proxies by the warps that load, which then wait for all their copies (110);
// loops over a tile's columns unrolled (406 instead of 317 for the batch of 64: the
// program is fetched again and again); the next part's Q before the last one's output,
// output through shared memory, one warp that walks for all: no gain.  Q in tensor
// memory with one S (128 us become 146, 209 become 234), or its half there with S tiles
// that overlap by half (within 4% either way); weights from the last maximum while the
// next is taken, and again where it grew (211 become 225; e4m3 136 become 158); the
// second half of S read under the first one's maximum (233 instead of 220 for heads
// of 64).
//
// Every wait has a limit; a role that runs into it sets MOE_DEVERR_TIMEOUT, and
// all leave.
#include <cuda_fp16.h>

#include "attn_tree.cuh"
#include "attn_tree_tc.cuh"

namespace moe {

constexpr uint64_t kTreeWaitNs = 2000000000ull;
constexpr int kLoadWarp = 4, kMmaWarp = 5, kReadyWarp = 6;  // and one more
static_assert(kTcThreads == 32 * (kReadyWarp + 2), "warps of a CTA");

template <int KV, int DP>
struct TcShape {
  using C = TcCfg<DP>;
  static constexpr int RING = 163840 / C::CTAS / (C::TILE * DP * 2);
  static constexpr int BUF = C::TILE * DP * 2;     // bytes of a tile
  static constexpr int PANEL = C::TILE * 128;      // of 64 columns of it
  static constexpr int QBLOCK = 128 * DP * 2;
  static constexpr int TMEM = DP == 256 ? 512 : 256;  // columns
  static constexpr int O = TMEM / 2;               // first of O's; S: from 0 and TILE on
  static constexpr int ES = kv_esize(KV);
  // warps that make ready: e4m3 tiles are work for two; else one of them loads values
  static constexpr int READY = KV == MOE_KV_E4M3 ? 2 : 1;
  static constexpr int CPR = DP * ES / 16;         // 16-byte chunks of a cached row
  static constexpr float LIFT = KV == MOE_KV_E4M3 ? kTreeLift : 0.0f;
  static constexpr float LAG = KV == MOE_KV_E4M3 ? 2.0f : 8.0f;
  // where e4m3 codes land: the last panels, or with one panel the second half of
  // each 32 rows' part of it
  static constexpr int PANELS = DP / 64;
  static constexpr int RAW = KV == MOE_KV_E4M3 ? (DP == 64 ? 0 : PANELS / 2) : 0;  // first panel
  static constexpr int LAND = KV == MOE_KV_E4M3 ? (DP == 64 ? 1 : PANELS / 2) : PANELS;
  static constexpr int LAND_ROW = KV == MOE_KV_E4M3 && DP == 64 ? 64 : 128;  // bytes of a row
  static constexpr uint32_t FMT = KV == MOE_KV_E4M3 ? 0 : 1;  // f16, bf16
};
// a logit's factor is not 0, so that a masked one's -inf stays that
constexpr float kTcLeast = 1.4e-45f;
constexpr int kSlots = 8;  // tiles whose live and non-finite tokens are kept

// What lies behind the tiles in shared memory
struct TcShared {
  uint64_t landed[10], full[10], empty[10], s_full[2], p_full[2], o_full[2], q_full, drain;
  TreeStart start;
  long long sums[33];
  uint32_t live[kSlots][2], wild[kSlots][2];  // bits by token
  uint32_t tmem;
  int abort;
};
static_assert(sizeof(TcShared) <= kTcShared, "shared memory of the kernel");

__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id,
                                          uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(id), "r"(acc)
      : "memory");
}
__device__ __forceinline__ bool tc_elect() {
  uint32_t one;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(one));
  return one != 0;
}
// A tile whose 64-column panels hold 128 bytes of each token, for a product over
// tokens: columns are the contiguous axis.  `panel`: bytes from one to the next
__device__ __forceinline__ uint64_t tc_desc_tokens(uint32_t saddr, uint32_t panel) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(panel >> 4) << 16;
  d |= static_cast<uint64_t>(1024u >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(2u) << 61;
  return d;
}
__device__ __forceinline__ void tc_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tc_st32(uint32_t taddr, const float (&v)[32]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t r[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(v[16 * h + i]);
    tc_st16(taddr + 16 * h, r);
  }
}
__device__ __forceinline__ void tc_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ uint4 tc_lds4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ void tc_sts4(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y),
               "r"(v.z), "r"(v.w)
               : "memory");
}
__device__ __forceinline__ uint32_t tc_f16x2(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
// two f32 operations an instruction
__device__ __forceinline__ uint64_t tc_pack(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 tc_unpack(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t tc_fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t tc_add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float tc_max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// four e4m3 codes as two pairs of f16: exact
__device__ __forceinline__ void tc_widen(uint32_t codes, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(codes));
}
// a pair of 16-bit numbers with those that are not finite replaced by 0; `wild`
// tells that there were some
template <uint32_t EXP>
__device__ __forceinline__ uint32_t tc_tame(uint32_t v, bool& wild) {
  const bool lo = (v & EXP) == EXP, hi = (v & (EXP << 16)) == (EXP << 16);
  wild |= lo || hi;
  return (lo ? 0 : v & 0xffffu) | (hi ? 0 : v & 0xffff0000u);
}
// byte of chunk c (16 bytes) of row r in a tile of 64-column panels, 128-byte swizzle
__device__ __forceinline__ uint32_t tc_chunk(int r, int c, int panel) {
  return (c >> 3) * panel + r * 128 + (((c & 7) ^ (r & 7)) << 4);
}

// byte where chunk c of cached row r lands
template <int KV, int DP>
__device__ __forceinline__ uint32_t tc_land(int r, int c) {
  using S = TcShape<KV, DP>;
  if constexpr (S::LAND_ROW == 64) return (r >> 5) * 4096 + 2048 + (r & 31) * 64 + c * 16;
  return tc_chunk(r, c + 8 * S::RAW, S::PANEL);
}
__device__ __forceinline__ void tc_tma4(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x,
                                        int y, int z, int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
}

template <int DP>
using TcWalk = TreeWalk<TcCfg<DP>::ROWS, TcCfg<DP>::TILE, TcCfg<DP>::END>;

// whether some row does not attend all of the tile at pos (bad pages aside)
template <int TILE>
__device__ __forceinline__ bool tc_masked(const TreeArgs& A, const TreeSpan& s, int pos) {
  const int lim = min(min(s.n, s.len - s.ctx), 64 * A.words);
  const int low = A.window > 0 ? s.ctx - max(0, A.window - max(0, lim)) : 0;
  return pos < low || pos + TILE > min(s.ctx, s.len);
}

// ------------------------------------------------------------ loads
// By TMA: a box is A.box tokens of a page and 64 columns, a lane has a box (all
// panels of it) of each tile.  The page ids of a tile are asked for a tile ahead.
// A warp takes 0.6 us to ask for a tile of four boxes: keys and values have one each
// where there is one to spare (keys, values: which this warp has).
template <int KV, int DP>
__device__ __forceinline__ void tc_tma_role(const TreeArgs& A, const CUtensorMap* k_map,
                                            const CUtensorMap* v_map, TcShared& sh, uint32_t ring,
                                            int lane, bool keys, bool values) {
  using S = TcShape<KV, DP>;
  constexpr int TILE = S::C::TILE, CH = TILE / 32;
  auto walk = tree_walk<S::C::ROWS, TILE, S::C::END>(A, sh.start);
  auto at = walk;
  bool ok = true, more = walk.next(A, at);
  uint32_t n = 0;  // tiles of the ring so far
  uint32_t asked = 0, phases = 0;  // bits by tile of the ring: this warp asked last, in which turn
  int slot = 0;
  const int box_shift = 31 - __clz(A.box), boxes = TILE >> box_shift;
  const int bytes = A.box * S::LAND * S::LAND_ROW;
  struct Place {
    int page, row;  // of this lane's box
    bool live;
  };
  auto want = [&](const TcWalk<DP>& p, int t) {
    Place w = {0, 0, false};
    const int pos = p.s.first + t * TILE + lane * A.box;
    if (lane < boxes && pos < p.s.len) {
      const int col = A.page_shift >= 0 ? pos >> A.page_shift : pos / A.page;
      w.row = pos - col * A.page;
      w.page = __ldg(A.table + p.b * A.table_stride + col);
      w.live = true;
    }
    return w;
  };
  auto ask = [&](bool kv, const Place& p, int kvh) {
    const int buf = static_cast<int>(n % S::RING);
    const uint32_t base = ring + buf * S::BUF, bar = smem_u32(&sh.landed[buf]);
    if (n >= S::RING && !__all_sync(0xffffffffu, mbar_wait(smem_u32(&sh.empty[buf]),
                                                           (n / S::RING - 1) & 1, kTreeWaitNs,
                                                           &sh.abort))) {
      atomicExch(&sh.abort, 1);
      return false;
    }
    const int count = __popc(__ballot_sync(0xffffffffu, p.live));
    if (lane == 0) mbar_arrive_expect_tx(bar, count * bytes);
    __syncwarp();
    asked |= 1u << buf;
    phases = (phases & ~(1u << buf)) | (n / S::RING & 1) << buf;
    if (p.live) {
      const int r = lane * A.box;
#pragma unroll
      for (int j = 0; j < S::LAND; ++j)
        tc_tma4(base + (S::LAND_ROW == 64 ? tc_land<KV, DP>(r, 0)
                                          : (j + S::RAW) * S::PANEL + r * 128),
                kv ? v_map : k_map, bar, j * (S::LAND_ROW / S::ES), p.row, kvh, p.page);
    }
    return true;
  };
  Place next = {0, 0, false};
  if (more) next = want(at, at.t0);
  while (more && ok) {
    const int kvh = at.head();
    auto after = at;
    bool goes_on = true;
    Place now = {0, 0, false}, before = now;
    for (int t = at.t0; ok && t <= at.t1; ++t) {
      before = now;
      if (t < at.t1) {
        now = next;
        now.live = now.live && now.page >= 0 && now.page < A.num_pages;
        if (t + 1 < at.t1) {
          next = want(at, t + 1);
        } else {
          goes_on = walk.next(A, after);
          if (goes_on) next = want(after, after.t0);
        }
        if (keys) {
          // which tokens there are, 32 a word
          const uint32_t there = __ballot_sync(0xffffffffu, now.live);
          if (lane < CH) {
            const int from = 32 * lane;
            uint32_t w = 0;
            if (A.box >= 32) {
              w = there >> (from >> box_shift) & 1u ? ~0u : 0u;
            } else {
#pragma unroll
              for (int b = 0; b < 32; b += 8)
                if (there >> (from + b >> box_shift) & 1u) w |= 0xffu << b;
            }
            const int left = at.s.len - (at.s.first + t * TILE + from);
            if (left < 32) w = left <= 0 ? 0 : w & ((1u << left) - 1);
            sh.live[slot][lane] = w;
          }
          slot = (slot + 1) % kSlots;
          __syncwarp();
          ok = ask(false, now, kvh);
        } else {
          asked &= ~(1u << n % S::RING);  // the other warp has it from here on
        }
        ++n;
      }
      if (t > at.t0) {
        if (ok && values) ok = ask(true, before, kvh);
        if (!values) asked &= ~(1u << n % S::RING);
        ++n;
      }
    }
    at = after;
    more = goes_on;
  }
  // nothing may be on its way to memory that the CTA gives up
  int never = 0;
  for (int i = 0; i < S::RING; ++i)
    if (asked >> i & 1u) mbar_wait(smem_u32(&sh.landed[i]), phases >> i & 1, kTreeWaitNs, &never);
}

// By cp.async, for pages that no box of eight tokens or more divides.  (A warp has
// few copies under way at a time: 1.6 us for 16 KB; the batch of 16 nodes takes 84 us
// in pages of 1, 4 or 5, bf16 and e4m3, and 64 in pages of 16, caches cold.)
template <int KV, int DP>
__device__ __forceinline__ void tc_load_role(const TreeArgs& A, TcShared& sh, uint32_t ring,
                                             int lane) {
  using S = TcShape<KV, DP>;
  constexpr int TILE = S::C::TILE, NW = TILE / 32;
  constexpr int CPR = S::CPR, RPI = 32 / CPR;  // rows at a time
  auto walk = tree_walk<S::C::ROWS, TILE, S::C::END>(A, sh.start);
  auto at = walk;
  bool ok = true, more = walk.next(A, at);
  uint32_t n = 0;  // tiles asked for
  int slot = 0;
  const int row0 = lane / CPR, chunk = lane % CPR;  // of this lane, of the first rows
  const bool real_chunk = chunk * 16 < A.dim * S::ES;

  // this lane's tokens (one of every 32): their pages, asked for a
  // tile ahead
  struct Want {
    int row[NW], page[NW];  // row in the page, -1: none
  };
  auto want = [&](const TcWalk<DP>& p, int t) {
    Want w;
#pragma unroll
    for (int i = 0; i < NW; ++i) {
      const int pos = p.s.first + t * TILE + 32 * i + lane;
      w.row[i] = -1;
      w.page[i] = 0;
      if (pos < p.s.len) {
        const int col = A.page_shift >= 0 ? pos >> A.page_shift : pos / A.page;
        w.row[i] = pos - col * A.page;
        w.page[i] = __ldg(A.table + p.b * A.table_stride + col);
      }
    }
    return w;
  };
  struct Place {
    long long off[NW];  // of this lane's tokens in the cache
    uint32_t mask[NW];  // which tokens are there
  };
  // ask for a tile of keys or values
  auto ask = [&](bool kv, const Place& p) {
    const int buf = static_cast<int>(n % S::RING);
    if (n >= S::RING && !__all_sync(0xffffffffu, mbar_wait(smem_u32(&sh.empty[buf]),
                                                           (n / S::RING - 1) & 1, kTreeWaitNs,
                                                           &sh.abort))) {
      atomicExch(&sh.abort, 1);
      return false;
    }
    const uint32_t base = ring + buf * S::BUF;
    const char* const from = (kv ? A.v : A.k) + chunk * 16;
#pragma unroll
    for (int j = 0; j < TILE / RPI; ++j) {
      const int r = j * RPI + row0;
      const long long o = __shfl_sync(0xffffffffu, p.off[j * RPI / 32], r & 31);
      const bool real = (p.mask[j * RPI / 32] >> (r & 31) & 1u) && real_chunk;
      tree_cp16(base + tc_land<KV, DP>(r, chunk), real ? from + o : A.k, real);
    }
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(
                     smem_u32(&sh.landed[buf]))
                 : "memory");
    if (lane == 0) mbar_arrive(smem_u32(&sh.landed[buf]));  // for what was told of the tile
    ++n;
    return true;
  };
  Want next = {};
  if (more) next = want(at, at.t0);
  while (more && ok) {
    const int kvh = at.head();
    auto after = at;
    bool goes_on = true;
    Place now = {}, before = {};
    for (int t = at.t0; ok && t <= at.t1; ++t) {
      before = now;
      if (t < at.t1) {
#pragma unroll
        for (int i = 0; i < NW; ++i) {
          const bool in = next.page[i] >= 0 && next.page[i] < A.num_pages;
          const bool live = next.row[i] >= 0 && in;
          now.off[i] = live ? next.page[i] * A.s_page + next.row[i] * A.s_token + kvh * A.s_head : 0;
          now.mask[i] = __ballot_sync(0xffffffffu, live);
          if (lane == 0) sh.live[slot][i] = now.mask[i];
        }
        slot = (slot + 1) % kSlots;
        __syncwarp();
        if (t + 1 < at.t1) {
          next = want(at, t + 1);
        } else {
          goes_on = walk.next(A, after);
          if (goes_on) next = want(after, after.t0);
        }
        ok = ask(false, now);
      }
      if (ok && t > at.t0) ok = ask(true, before);
    }
    at = after;
    more = goes_on;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// What has landed is made ready for the products: e4m3 codes are widened, values
// that are not finite tamed where masks apply, and the tile passes from the
// proxy that it was written through to the one that the products read through.
// (A thread with copies under way would wait for them at that fence: the warps
// that load do not take it.)
template <int KV, int DP>
__device__ __forceinline__ void tc_ready_role(const TreeArgs& A, TcShared& sh, uint32_t ring,
                                              int warp, int lane) {
  using S = TcShape<KV, DP>;
  constexpr int TILE = S::C::TILE, TPW = TILE / S::READY, WORDS = TPW / 32;
  constexpr int CPR = S::CPR, RPI = 32 / CPR;
  auto walk = tree_walk<S::C::ROWS, TILE, S::C::END>(A, sh.start);
  auto at = walk;
  uint32_t n = 0;
  int slot = 0;
  const int row0 = lane / CPR, chunk = lane % CPR;
  auto ready = [&](bool kv, int t) {
    const int buf = static_cast<int>(n % S::RING);
    if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&sh.landed[buf]), n / S::RING & 1, kTreeWaitNs,
                                           &sh.abort))) {
      atomicExch(&sh.abort, 1);
      return false;
    }
    const uint32_t base = ring + buf * S::BUF;
    const bool tame = kv && tc_masked<TILE>(A, at.s, at.s.first + t * TILE);
    uint32_t wild_rows[WORDS] = {};
    // tokens that are not there: whatever lies in their rows must not count as values
    uint32_t there[WORDS];
    bool gaps = false;
#pragma unroll
    for (int i = 0; i < WORDS; ++i) {
      there[i] = kv ? *reinterpret_cast<const volatile uint32_t*>(&sh.live[slot][warp * WORDS + i])
                    : ~0u;
      gaps = gaps || there[i] != ~0u;
    }
    const bool care = tame || gaps;
    if constexpr (KV == MOE_KV_E4M3) {
      uint4 raw[TPW / RPI];
#pragma unroll
      for (int j = 0; j < TPW / RPI; ++j)
        raw[j] = tc_lds4(base + tc_land<KV, DP>(warp * TPW + j * RPI + row0, chunk));
      __syncwarp();  // the codes lie where the warp's rows are written
#pragma unroll
      for (int j = 0; j < TPW / RPI; ++j) {
        const int r = warp * TPW + j * RPI + row0;
        uint4 lo, hi;
        tc_widen(raw[j].x, lo.x, lo.y);
        tc_widen(raw[j].y, lo.z, lo.w);
        tc_widen(raw[j].z, hi.x, hi.y);
        tc_widen(raw[j].w, hi.z, hi.w);
        tc_sts4(base + tc_chunk(r, 2 * chunk, S::PANEL), lo);
        tc_sts4(base + tc_chunk(r, 2 * chunk + 1, S::PANEL), hi);
      }
    }
    if (care) {  // a few tiles of a unit: a short program rather than a fast one
      constexpr int PER = KV == MOE_KV_E4M3 ? 2 : 1;  // chunks of this lane in a row
#pragma unroll 1
      for (int j = 0; j < TPW / RPI * PER; ++j) {
        const int in = j / PER * RPI + row0;
        const uint32_t to = base + tc_chunk(warp * TPW + in, chunk * PER + j % PER, S::PANEL);
        const uint32_t bit = 1u << (in & 31);
        if (!((WORDS > 1 && in >= 32 ? there[WORDS - 1] : there[0]) & bit)) {
          tc_sts4(to, make_uint4(0, 0, 0, 0));
          continue;
        }
        if (!tame) continue;
        constexpr uint32_t EXP = KV == MOE_KV_E4M3 ? 0x7c00u : 0x7f80u;
        uint4 v = tc_lds4(to);
        bool wild = false;
        v.x = tc_tame<EXP>(v.x, wild);
        v.y = tc_tame<EXP>(v.y, wild);
        v.z = tc_tame<EXP>(v.z, wild);
        v.w = tc_tame<EXP>(v.w, wild);
        if (wild) {
          if (WORDS > 1 && in >= 32) wild_rows[WORDS - 1] |= bit;
          else wild_rows[0] |= bit;
          tc_sts4(to, v);
        }
      }
    }
    if (tame) {
#pragma unroll
      for (int i = 0; i < WORDS; ++i) {
        const uint32_t w = __reduce_or_sync(0xffffffffu, wild_rows[i]);
        if (lane == 0) sh.wild[slot][warp * WORDS + i] = w;
      }
    }
    if (kv) slot = (slot + 1) % kSlots;
    // (what TMA has written needs none)
    if (KV == MOE_KV_E4M3 || A.box == 0 || care) fence_proxy_async_shared();
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&sh.full[buf]));
    ++n;
    return true;
  };
  while (walk.next(A, at)) {
    for (int t = at.t0; t <= at.t1; ++t) {
      if (t < at.t1 && !ready(false, t)) return;
      if (t > at.t0 && !ready(true, t - 1)) return;
    }
  }
}

// ------------------------------------------------------------ products
// The whole warp keeps step, so that descriptors are the warp's and not a lane's,
// and one lane issues.
template <int KV, int DP>
__device__ __forceinline__ void tc_mma_role(const TreeArgs& A, TcShared& sh, uint32_t qs,
                                            uint32_t ring) {
  using S = TcShape<KV, DP>;
  constexpr int TILE = S::C::TILE;
  constexpr uint32_t kS = idesc_make(S::FMT, 128, TILE);
  constexpr uint32_t kO = idesc_make(S::FMT, 128, DP) | (1u << 16);  // V: columns contiguous
  auto walk = tree_walk<S::C::ROWS, TILE, S::C::END>(A, sh.start);
  auto at = walk;
  const uint32_t tmem = __shfl_sync(0xffffffffu, sh.tmem, 0);
  const uint64_t qd = sdesc_sw128(qs), kd = sdesc_sw128(ring), vd = tc_desc_tokens(ring, S::PANEL);
  const uint32_t full = smem_u32(sh.full), empty = smem_u32(sh.empty), s_full = smem_u32(sh.s_full),
                 p_full = smem_u32(sh.p_full), o_full = smem_u32(sh.o_full);
  uint32_t buf = 0, turn = 0;  // the ring's next tile, and how often the ring has gone round
  uint32_t q = 0, parts = 0;   // tiles of weights, and parts before
  bool ok = true;
  auto wait = [&](uint32_t bar, uint32_t phase) {
    ok = ok && __all_sync(0xffffffffu, mbar_wait(bar, phase & 1, kTreeWaitNs, &sh.abort));
    return ok;
  };
  auto used = [&] {  // the tile at buf
    if (++buf == S::RING) {
      buf = 0;
      ++turn;
    }
  };
  while (ok && walk.next(A, at)) {
    const uint32_t tiles = at.t1 - at.t0;
    if (!wait(smem_u32(&sh.q_full), parts++)) break;
    // t: S of tile t, then O with the weights of the one before
    for (uint32_t t = 0; ok && t <= tiles; ++t) {
      if (t < tiles) {
        const uint32_t i = q + t, b = i & 1;
        // this S holds the weights of the tile before last: used up
        if (i >= 2 && !wait(o_full + 8 * b, i / 2 - 1)) break;
        if (!wait(full + 8 * buf, turn)) break;
        tc_fence_after();
        const uint64_t k = kd + (buf * S::BUF >> 4);
        if (tc_elect()) {
#pragma unroll
          for (int ks = 0; ks < DP / 16; ++ks)
            mma_issue<1>(tmem + b * TILE, qd + (ks / 4 * 16384 + ks % 4 * 32 >> 4),
                         k + (ks / 4 * S::PANEL + ks % 4 * 32 >> 4), kS, ks > 0);
          mma_commit(s_full + 8 * b);
          mma_commit(empty + 8 * buf);
        }
        __syncwarp();
        used();
      }
      if (t == 0) continue;
      const uint32_t i = q + t - 1, b = i & 1;
      if (!wait(full + 8 * buf, turn) || !wait(p_full + 8 * b, i / 2)) break;
      tc_fence_after();
      const uint64_t v = vd + (buf * S::BUF >> 4);
      if (tc_elect()) {
#pragma unroll
        for (int ks = 0; ks < TILE / 16; ++ks)
          tc_mma_ts(tmem + S::O, tmem + b * TILE + 8 * ks, v + (ks * 2048 >> 4), kO,
                    t > 1 || ks > 0);
        mma_commit(o_full + 8 * b);
        mma_commit(empty + 8 * buf);
      }
      __syncwarp();
      used();
    }
    q += tiles;
  }
  if (!ok) {
    atomicExch(&sh.abort, 1);
    // nothing of this CTA's may be under way when its memory goes
    if (tc_elect()) mma_commit(smem_u32(&sh.drain));
    __syncwarp();
    int never = 0;
    mbar_wait(smem_u32(&sh.drain), 0, kTreeWaitNs, &never);
  }
}

// ------------------------------------------------------------ softmax
template <int KV, int DP>
__device__ __forceinline__ void tc_softmax_role(const TreeArgs& A, TcShared& sh, uint32_t qs,
                                                int warp, int lane) {
  using S = TcShape<KV, DP>;
  constexpr int TILE = S::C::TILE, ROWS = S::C::ROWS;
  const int r = warp * 32 + lane;  // row of the block
  auto walk = tree_walk<ROWS, TILE, S::C::END>(A, sh.start);
  auto at = walk;
  const uint32_t tmem = sh.tmem + (static_cast<uint32_t>(warp * 32) << 16);
  const uint32_t t_o = tmem + S::O;
  uint32_t seq = 0;  // tiles before this part
  bool ok = true;
  auto wait = [&](uint64_t* bar, uint32_t phase) {
    ok = mbar_wait(smem_u32(bar), phase & 1, kTreeWaitNs, &sh.abort);
    return __all_sync(0xffffffffu, ok);
  };
  // the product with the weights of tile q.  (A barrier tells a phase from the one
  // before it only, and two products may be under way: a barrier for each S)
  auto wait_o = [&](uint32_t q) { return wait(&sh.o_full[q & 1], q / 2); };
  while (walk.next(A, at)) {
    const TreeSpan& s = at.s;
    const int kvh = at.head(), r0 = at.block() * ROWS;
    const int rows = min(ROWS, s.use * A.group - r0);
    const bool mine = r < rows;
    const int R = r0 + min(r, rows - 1), node = R / A.group, h = kvh * A.group + R - node * A.group;
    const long long row = s.row0 + node;
    // a warp whose rows are all beyond the block's only keeps step
    const bool idle = warp * 32 >= rows;
    const TreeMask mask = tree_mask(A, s, node);
    float sl = A.scale_log2, v_mul = 1.0f;
    if constexpr (KV == MOE_KV_E4M3) {
      sl *= A.k_scale[kvh];
      v_mul = A.v_scale[kvh];
    }
    // ---- the row of Q; a negative scale turns its sign instead of the logits', so
    // that the largest product is the largest logit
    float mul = 1.0f;
    {
      const uint32_t sign = sl < 0.0f ? 0x80008000u : 0u;
      const uint4* const q = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(A.q) +
                                                            row * A.q_n + h * A.q_h);
      constexpr int HALF = DP / 8 < 16 ? DP / 8 : 16;  // chunks at a time
      float inv = 1.0f;
      if constexpr (KV == MOE_KV_E4M3) {
        // as f16, scaled by a power of two that brings the largest into [1, 2):
        // bf16 has 8 bits and f16 11, only what lies below 2^-17 of it is rounded
        float big = 0.0f;
#pragma unroll
        for (int c = 0; c < DP / 8; ++c) {
          uint4 v = make_uint4(0, 0, 0, 0);
          if (mine && c * 8 < A.dim) v = __ldg(q + c);
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            big = fmaxf(big, fmaxf(fabsf(__uint_as_float(w[e] << 16)),
                                   fabsf(__uint_as_float(w[e] & 0xffff0000u))));
        }
        const int e = min(max(static_cast<int>(__float_as_uint(big) >> 23), 1), 253);
        mul = __uint_as_float(static_cast<uint32_t>(e) << 23);
        inv = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
      }
#pragma unroll 1
      for (int c0 = 0; c0 < DP / 8; c0 += HALF) {
        uint4 v[HALF];
#pragma unroll
        for (int c = 0; c < HALF; ++c) {
          v[c] = make_uint4(0, 0, 0, 0);
          if (mine && (c0 + c) * 8 < A.dim) v[c] = __ldg(q + c0 + c);
        }
#pragma unroll
        for (int c = 0; c < HALF; ++c) {
          uint32_t w[4] = {v[c].x ^ sign, v[c].y ^ sign, v[c].z ^ sign, v[c].w ^ sign};
          if constexpr (KV == MOE_KV_E4M3) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              w[e] = tc_f16x2(__uint_as_float(w[e] << 16) * inv,
                              __uint_as_float(w[e] & 0xffff0000u) * inv);
          }
          tc_sts4(qs + tc_chunk(r, c0 + c, 16384), make_uint4(w[0], w[1], w[2], w[3]));
        }
      }
      fence_proxy_async_shared();
      mbar_arrive(smem_u32(&sh.q_full));
    }
    const float f0 = fabsf(sl) * mul, f = f0 < kTcLeast ? kTcLeast : f0;  // of logits, in base 2
    const int low = tree_low(A, s, mask, node);
    const uint32_t tiles = at.t1 - at.t0;
    float m = -INFINITY, sum = 0.0f;
    for (uint32_t i = 0; i < tiles; ++i) {
      const int pos = s.first + (at.t0 + static_cast<int>(i)) * TILE;
      const uint32_t q = seq + i, b = q & 1, t_s = tmem + b * TILE;
      if (!wait(&sh.s_full[b], q / 2)) goto out;
      if (idle) {
        mbar_arrive(smem_u32(&sh.p_full[b]));
        continue;
      }
      tc_fence_after();
      float v[2][32];
      tmem_ld32(t_s, v[0]);
      tmem_ld32(t_s + 32, v[1]);
      const int slot = static_cast<int>(q % kSlots);
      const volatile uint32_t* const live = sh.live[slot];
      uint32_t word[2] = {live[0], live[1]};
      const bool masked = tc_masked<TILE>(A, s, pos);
      const bool all = !masked && (word[0] & word[1]) == ~0u;  // (the same for all rows)
      bool any = true;
      tmem_wait_ld(v[0], v[1]);
      if (!all) {  // logits that do not count become -inf
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const uint32_t want = tree_attends(s, mask, low, pos + 32 * c);
          // told of here, where it is known that a row attends the token: pages that all
          // rows have left behind may be gone
          if ((want & ~word[c]) && A.err) atomicOr(A.err, MOE_DEVERR_BAD_PAGE);
          word[c] &= want;
#pragma unroll
          for (int j = 0; j < 32; ++j) v[c][j] = word[c] >> j & 1u ? v[c][j] : -INFINITY;
        }
        any = (word[0] | word[1]) != 0;
      }
      float x[4] = {v[0][0], v[0][1], v[1][0], v[1][1]};
#pragma unroll
      for (int j = 2; j < 32; j += 4) {
        x[0] = tc_max3(x[0], v[0][j], v[0][j + 1]);
        x[2] = tc_max3(x[2], v[1][j], v[1][j + 1]);
        if (j + 2 < 32) {
          x[1] = tc_max3(x[1], v[0][j + 2], v[0][j + 3]);
          x[3] = tc_max3(x[3], v[1][j + 2], v[1][j + 3]);
        }
      }
      float top = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
      top = top == -INFINITY ? top : top * f;
      const bool grow = top > m + (S::LIFT + S::LAG);
      float keep = 1.0f;
      if (grow) {
        const float to = top - S::LIFT;
        keep = tree_ex2(m - to);
        m = to;
        sum *= keep;
      }
      // from here on the row has tokens, if only of logits -inf: m says so
      if (any) m = fmaxf(m, -FLT_MAX);
      const float ref = m == -INFINITY ? 0.0f : m;
      // (nothing attended: -inf stays that, whatever the scale, a NaN of e4m3 among them)
      const float by = KV == MOE_KV_E4M3 && !any ? 1.0f : f;
      const uint64_t f2 = tc_pack(by, by), ref2 = tc_pack(-ref, -ref);
      uint64_t part[2] = {0, 0};
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t p[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          float2 w = tc_unpack(tc_fma2(tc_pack(v[c][2 * j], v[c][2 * j + 1]), f2, ref2));
          w.x = tree_ex2(w.x);
          w.y = tree_ex2(w.y);
          part[j & 1] = tc_add2(part[j & 1], tc_pack(w.x, w.y));
          p[j] = KV == MOE_KV_E4M3 ? tc_f16x2(w.x, w.y) : tree_bf16x2(w.x, w.y);
        }
        tc_st16(t_s + 16 * c, p);
      }
      const float2 added = tc_unpack(tc_add2(part[0], part[1]));
      sum += added.x + added.y;
      if (i > 0 && __any_sync(0xffffffffu, grow)) {
        if (!wait_o(q - 1)) goto out;
        tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < DP; c += 32) {
          float o[32];
          tmem_ld32(t_o + c, o);
          tmem_wait_ld(o);
#pragma unroll
          for (int j = 0; j < 32; ++j) o[j] *= keep;
          tc_st32(t_o + c, o);
        }
      }
      tc_wait_st();
      tc_fence_before();
      mbar_arrive(smem_u32(&sh.p_full[b]));
      if (masked) {
        // values that are not finite: what they leave in the rows that attend them
        // (told before the values' barrier, which this product has waited for)
        if (!wait_o(q)) goto out;
        tc_fence_after();
        const volatile uint32_t* const wild = sh.wild[slot];
        if (wild[0] | wild[1]) {
#pragma unroll 1
          for (int d0 = 0; d0 < DP; d0 += 32) {
            float o[32];
            tmem_ld32(t_o + d0, o);
            tmem_wait_ld(o);
#pragma unroll 1
            for (int c = 0; c < 2; ++c) {
              uint32_t left = wild[c] & word[c];
              while (left) {
                const int tok = pos + 32 * c + __ffs(left) - 1;
                left &= left - 1;
                const int col = A.page_shift >= 0 ? tok >> A.page_shift : tok / A.page;
                const char* const from = A.v + A.table[at.b * A.table_stride + col] * A.s_page +
                                         (tok - col * A.page) * A.s_token + kvh * A.s_head;
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                  if (d0 + j >= A.dim) continue;
                  float y;
                  if constexpr (KV == MOE_KV_E4M3) {
                    const uint8_t e = *reinterpret_cast<const uint8_t*>(from + d0 + j);
                    y = (e & 0x7f) == 0x7f ? __uint_as_float(0x7fffffffu) : 0.0f;
                  } else {
                    y = __uint_as_float(
                        static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(from + 2 * (d0 + j)))
                        << 16);
                    if (fabsf(y) <= FLT_MAX) y = 0.0f;
                  }
                  o[j] += y;
                }
              }
            }
            tc_st32(t_o + d0, o);
          }
          tc_wait_st();
          tc_fence_before();
        }
      }
    }
    seq += tiles;
    if (!wait_o(seq - 1)) goto out;
    tc_fence_after();
    // ---- the part's end
    const bool whole = at.t0 == 0 && at.t1 == at.nt;
    const float inv = m == -INFINITY ? 0.0f : v_mul / sum;
    const long long part = 2ll * blockIdx.x + (at.t0 == 0 ? 0 : 1);
#pragma unroll 1
    for (int d = 0; !idle && d < DP; d += 32) {
      float o[32];
      tmem_ld32(t_o + d, o);
      tmem_wait_ld(o);
      if (!mine) continue;
      if (whole) {
#pragma unroll
        for (int j = 0; j < 32; j += 8)
          if (d + j < A.dim)
            *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(A.out) + row * A.o_n + h * A.o_h +
                                      d + j) =
                make_uint4(tree_bf16x2(o[j] * inv, o[j + 1] * inv),
                           tree_bf16x2(o[j + 2] * inv, o[j + 3] * inv),
                           tree_bf16x2(o[j + 4] * inv, o[j + 5] * inv),
                           tree_bf16x2(o[j + 6] * inv, o[j + 7] * inv));
      } else {
#pragma unroll
        for (int j = 0; j < 32; j += 4)
          *reinterpret_cast<float4*>(A.part_o + (part * ROWS + r) * DP + d + j) =
              make_float4(o[j], o[j + 1], o[j + 2], o[j + 3]);
      }
    }
    if (mine) {
      if (!whole) A.part_ml[part * ROWS + r] = make_float2(m, sum);
      else if (A.lse) A.lse[row * A.Hq + h] = tree_lse<KV>(m, sum);
    }
    if (r == 0 && at.t1 < at.nt) tree_record(A, sh.start, at);
    tc_fence_before();
  }
out:
  if (!ok) {
    atomicExch(&sh.abort, 1);
    if (A.err) atomicOr(A.err, MOE_DEVERR_TIMEOUT);
  }
}

template <int KV, int DP>
__global__ void __launch_bounds__(kTcThreads, TcCfg<DP>::CTAS)
    tree_tc_kernel(const __grid_constant__ TreeArgs A, const __grid_constant__ CUtensorMap k_map,
                   const __grid_constant__ CUtensorMap v_map) {
  using S = TcShape<KV, DP>;
  extern __shared__ __align__(1024) uint8_t tc_smem[];
  const uint32_t qs = smem_u32(tc_smem), ring = qs + S::QBLOCK;
  TcShared& sh = *reinterpret_cast<TcShared*>(tc_smem + S::QBLOCK + S::RING * S::BUF);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0 && A.box) {
    prefetch_tmap(&k_map);
    prefetch_tmap(&v_map);
  }
  pdl_wait();
  if (qs & 1023) {  // (a CTA's shared memory begins at a multiple of that)
    if (tid == 0) A.info[blockIdx.x] = make_int4(0, 0, 0, 0);
    if (tid == 0 && A.err) atomicOr(A.err, MOE_DEVERR_TIMEOUT);
    return;
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(&sh.tmem), S::TMEM);
    tmem_relinquish();
  }
  if (tid == 0) {
    for (int i = 0; i < S::RING; ++i) {
      mbar_init(smem_u32(&sh.landed[i]), A.box ? 1 : 33);
      mbar_init(smem_u32(&sh.full[i]), S::READY);
      mbar_init(smem_u32(&sh.empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&sh.s_full[i]), 1);
      mbar_init(smem_u32(&sh.p_full[i]), 128);
      mbar_init(smem_u32(&sh.o_full[i]), 1);
    }
    mbar_init(smem_u32(&sh.q_full), 128);
    mbar_init(smem_u32(&sh.drain), 1);
    fence_mbar_init();
    sh.abort = 0;
  }
  tc_fence_before();
  pdl_trigger();
  tree_begin<S::C::ROWS, S::C::TILE, S::C::END>(A, &sh.start, sh.sums);
  tc_fence_after();
  if (warp < kLoadWarp) {
    tc_softmax_role<KV, DP>(A, sh, qs, warp, lane);
  } else if (warp == kMmaWarp) {
    tc_mma_role<KV, DP>(A, sh, qs, ring);
  } else if (warp >= kReadyWarp + 2 - S::READY) {
    tc_ready_role<KV, DP>(A, sh, ring, warp - (kReadyWarp + 2 - S::READY), lane);
  } else if (A.box) {
    tc_tma_role<KV, DP>(A, &k_map, &v_map, sh, ring, lane, warp == kLoadWarp,
                        S::READY == 2 || warp == kReadyWarp);
  } else if (warp == kLoadWarp) {
    tc_load_role<KV, DP>(A, sh, ring, lane);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(sh.tmem, S::TMEM);
}

// ------------------------------------------------------------ host
typedef CUresult (*TreeEncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                 const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                 const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
static TreeEncodeFn tree_encode_fn() {
  static const TreeEncodeFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    const bool ok = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000,
                                                     cudaEnableDefault, &q) == cudaSuccess &&
                    q == cudaDriverEntryPointSuccess;
    return ok ? reinterpret_cast<TreeEncodeFn>(p) : nullptr;
  }();
  return fn;
}

// The maps of keys and values for boxes of 64 columns by `box` tokens of a page;
// false where there are none of these pages and strides
template <int KV, int DP>
static bool tree_maps(const TreeArgs& a, int box, CUtensorMap* maps) {
  using S = TcShape<KV, DP>;
  const TreeEncodeFn fn = tree_encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(a.dim), static_cast<cuuint64_t>(a.page),
                              static_cast<cuuint64_t>(a.heads),
                              static_cast<cuuint64_t>(a.num_pages)};
  const cuuint64_t row = static_cast<cuuint64_t>(a.dim) * S::ES;  // where an axis has one element
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(a.s_token),
                                 a.heads > 1 ? static_cast<cuuint64_t>(a.s_head) : row,
                                 a.num_pages > 1 ? static_cast<cuuint64_t>(a.s_page) : row};
  const cuuint32_t shape[4] = {S::LAND_ROW / S::ES, static_cast<cuuint32_t>(box), 1, 1};
  const cuuint32_t ones[4] = {1, 1, 1, 1};
  for (int i = 0; i < 3; ++i)
    if (strides[i] < row || strides[i] >= 1ull << 40) return false;
  for (int i = 0; i < 2; ++i)
    if (fn(maps + i, KV == MOE_KV_E4M3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                       : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
           4, const_cast<char*>(i ? a.v : a.k), dims, strides, shape, ones,
           CU_TENSOR_MAP_INTERLEAVE_NONE,
           S::LAND_ROW == 64 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B,
           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return false;
  return true;
}

template <int KV, int DP>
static cudaError_t launch_tc(TreeArgs a, int ctas, cudaStream_t st) {
  using S = TcShape<KV, DP>;
  constexpr int SMEM = S::QBLOCK + S::RING * S::BUF + kTcShared;
  static_assert(S::C::CTAS * (SMEM + 1024) <= 228 * 1024, "shared memory of an SM");
  auto* kern = tree_tc_kernel<KV, DP>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), SMEM, done);
  if (e != cudaSuccess) return e;
  // a box: the largest power of two that divides a page, up to what lands in one
  // piece; tiles begin at multiples of it
  constexpr int kMost = S::LAND_ROW == 64 ? 32 : S::C::TILE;
  int box = a.page & -a.page;
  box = box < kMost ? box : kMost;
  CUtensorMap maps[2] = {};
  a.box = box >= 8 && tree_maps<KV, DP>(a, box, maps) ? box : 0;
  e = launch_chained(kern, dim3(ctas), dim3(kTcThreads), SMEM, st, a, maps[0], maps[1]);
  if (e != cudaSuccess) return e;
  return launch_chained(tree_join_kernel<KV, DP, S::C::ROWS>, dim3(ctas, kTreeJoinBlocks),
                        dim3(32 * kTreeJoinWarps), 0, st, a);
}

cudaError_t launch_tree_tc(int kv, int dp, const TreeArgs& a, int ctas, cudaStream_t st) {
  if (kv == MOE_KV_BF16)
    return dp == 64    ? launch_tc<MOE_KV_BF16, 64>(a, ctas, st)
           : dp == 128 ? launch_tc<MOE_KV_BF16, 128>(a, ctas, st)
                       : launch_tc<MOE_KV_BF16, 256>(a, ctas, st);
  return dp == 64    ? launch_tc<MOE_KV_E4M3, 64>(a, ctas, st)
         : dp == 128 ? launch_tc<MOE_KV_E4M3, 128>(a, ctas, st)
                     : launch_tc<MOE_KV_E4M3, 256>(a, ctas, st);
}

}  // namespace moe
