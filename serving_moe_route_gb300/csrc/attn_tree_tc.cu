// attn_tree_tc.cu -- moe_attn_tree on the 5th-generation tensor cores, for bf16
// and e4m3 caches.
//
// S = Q K^T and O += P V with tcgen05.mma on tiles of TILE tokens, 128 rows of
// (node, query head) a block.  A CTA has one block per SM and two lanes, each
// with a logit tile S, an accumulator O in tensor memory and a warpgroup that
// owns its softmax, a row a thread:
//   a unit of up to 128 rows   the lanes take its tiles in turn and join at its
//                              end, so that one's products run under the other's
//                              softmax;
//   a unit of up to 256 rows   each lane has 128 of them and both use every tile:
//                              a cached byte is used twice as often.
// head_dim above 128 leaves tensor memory for one O: one lane, two S tiles of
// half the size.
//
//   loads    one warp fills a ring of key and value tiles by TMA, as far ahead as
//            it reaches, across unit borders (pages that 8 does not divide: two
//            warps, by cp.async).  Four others make ready what has landed: e4m3
//            codes lie in the half of their tile that the same warp will write,
//            and are widened to f16, which holds them exactly.
//   softmax  one pass with a reference m and the sum l of a row in fp32 (base 2);
//            O is rescaled only when a logit lies LAG above the one that m was
//            taken from.  P is rounded to bf16 (f16 for e4m3 caches) into the
//            columns of S that it has been read from; l adds the weights before
//            that.  f16 weights are lifted to 2^LIFT, which keeps 11 bits down to
//            2^-27 of the largest.
//   masks    Only tiles that some row does not wholly attend look at masks.  Their
//            weights are 0, but 0 times a value that is not finite is not: such
//            values are replaced by 0 in the tile, and added to O for the rows
//            that do attend them.
//
// Every wait has a limit; a role that runs into it sets MOE_DEVERR_TIMEOUT, and
// all leave.
#include <cuda_fp16.h>

#include "attn_tree.cuh"
#include "attn_tree_tc.cuh"

namespace moe {

constexpr uint64_t kTreeWaitNs = 2000000000ull;
constexpr int kLoadWarps = 2, kReadyWarps = 4, kMmaWarp = 8 + kLoadWarps + kReadyWarps;
static_assert(kTcThreads == 32 * (kMmaWarp + 1), "two softmax warpgroups, loads, products");

template <int KV, int DP>
struct TcShape {
  using C = TcCfg<DP>;
  static constexpr int RING = 163840 / (C::TILE * DP * 2);
  static constexpr int BUF = C::TILE * DP * 2;     // bytes of a tile
  static constexpr int PANEL = C::TILE * 128;      // of 64 columns of it
  static constexpr int QBLOCK = 128 * DP * 2;
  static constexpr int NB = C::LANES == 1 ? 2 : 1; // S tiles of a lane
  static constexpr int ES = kv_esize(KV);
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
// a logit's factor is not 0, so that -inf stays -inf
constexpr float kTcLeast = 1e-37f;
constexpr int kSlots = 8;  // tiles whose live and non-finite tokens are kept

// The second block of Q's memory where a unit has one block only: what the
// lanes that take turns tell each other
struct TcTurns {
  float m[2][128], sum[2][128], q_mul[128];
};
// What lies behind the tiles in shared memory
struct TcShared {
  uint64_t landed[10], full[10], empty[10], s_full[2], p_full[2], o_full[2], q_full[2], join[2], drain;
  TreeStart start;
  long long sums[kTcThreads / 32];
  uint8_t live[kSlots][16], wild[kSlots][16];  // bits by token
  uint32_t tmem;
  int abort;
};
static_assert(sizeof(TcShared) <= kTcShared, "shared memory of the kernel");
static_assert(sizeof(TcTurns) <= 128 * 64 * 2, "a block of Q");

__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id,
                                          uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(id), "r"(acc)
      : "memory");
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
__device__ __forceinline__ void tc_cp16(uint32_t dst, const void* src, bool real) {
  // a chunk that is not real is filled with zeros and nothing is read
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(real ? 16 : 0)
               : "memory");
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

// Tiles lie in the ring in the order in which they are first used.  Where one lane
// has all of a unit's rows, the next tile's keys come before a tile's values:
// K0 K1 V0 K2 V1 ...  Else both lanes use each tile: K0 V0 K1 V1 ...
template <int DP>
__device__ __forceinline__ bool tc_pair(const TreeArgs& A, const TcWalk<DP>& at) {
  const int blocks = at.units / A.heads;
  return TcCfg<DP>::LANES == 2 && at.s.use * A.group - at.x % blocks * TcCfg<DP>::ROWS > 128;
}
// ------------------------------------------------------------ loads
// By TMA, one warp: a box is A.box tokens of a page and 64 columns, a lane has a
// box (or two panels of it) of each tile.  The page ids of a tile are asked for a
// tile ahead.
template <int KV, int DP>
__device__ __forceinline__ void tc_tma_role(const TreeArgs& A, const CUtensorMap* k_map,
                                            const CUtensorMap* v_map, TcShared& sh, uint32_t ring,
                                            int lane) {
  using S = TcShape<KV, DP>;
  constexpr int TILE = S::C::TILE, CH = TILE / 32;
  auto walk = tree_walk<S::C::ROWS, TILE, S::C::END>(A, sh.start);
  auto at = walk;
  bool bad_page = false, ok = true, more = walk.next(A, at);
  uint32_t n = 0;  // tiles asked for
  int slot = 0;
  const int boxes = TILE / A.box;
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
    if (n >= S::RING && !__all_sync(0xffffffffu, mbar_wait(smem_u32(&sh.empty[buf]),
                                                           (n / S::RING - 1) & 1, kTreeWaitNs,
                                                           &sh.abort))) {
      atomicExch(&sh.abort, 1);
      return false;
    }
    const uint32_t base = ring + buf * S::BUF, bar = smem_u32(&sh.landed[buf]);
    const int count = __popc(__ballot_sync(0xffffffffu, p.live));
    if (lane == 0) mbar_arrive_expect_tx(bar, count * bytes);
    __syncwarp();
    if (p.live) {
      const int r = lane * A.box;
#pragma unroll
      for (int j = 0; j < S::LAND; ++j)
        tc_tma4(base + (S::LAND_ROW == 64 ? tc_land<KV, DP>(r, 0)
                                          : (j + S::RAW) * S::PANEL + r * 128),
                kv ? v_map : k_map, bar, j * (S::LAND_ROW / S::ES), p.row, kvh, p.page);
    }
    ++n;
    return true;
  };
  Place next = {0, 0, false};
  if (more) next = want(at, at.t0);
  while (more && ok) {
    const int kvh = at.x / (at.units / A.heads);
    const bool late = !tc_pair<DP>(A, at);
    auto after = at;
    bool goes_on = true;
    Place now = {0, 0, false}, before = now;
    for (int t = at.t0; ok && t < at.t1 + late; ++t) {
      before = now;
      if (t < at.t1) {
        now = next;
        if (now.live && (now.page < 0 || now.page >= A.num_pages)) {
          bad_page = true;
          now.live = false;
        }
        // which tokens there are, 32 a word
        const uint32_t there = __ballot_sync(0xffffffffu, now.live);
        if (lane < CH) {
          uint32_t w = 0;
          const int from = 32 * lane;
          for (int b = from / A.box; b * A.box < from + 32; ++b)
            if (there >> b & 1u)
              w |= A.box >= 32 ? ~0u : ((1u << A.box) - 1) << (b * A.box - from);
          const int left = at.s.len - (at.s.first + t * TILE + from);
          if (left < 32) w = left <= 0 ? 0 : w & ((1u << left) - 1);
          *reinterpret_cast<uint32_t*>(&sh.live[slot][4 * lane]) = w;
        }
        slot = (slot + 1) % kSlots;
        __syncwarp();
        if (t + 1 < at.t1) {
          next = want(at, t + 1);
        } else {
          goes_on = walk.next(A, after);
          if (goes_on) next = want(after, after.t0);
        }
        ok = ask(false, now, kvh);
      }
      if (ok && !(late && t == at.t0)) ok = ask(true, late ? before : now, kvh);
    }
    at = after;
    more = goes_on;
  }
  if (bad_page && A.err) atomicOr(A.err, MOE_DEVERR_BAD_PAGE);
}

// By cp.async, two warps, for pages that no box of eight tokens or more divides.
// A warp has few copies under way at a time: 1.6 us for a tile of 32 KB.
template <int KV, int DP>
__device__ __forceinline__ void tc_load_role(const TreeArgs& A, TcShared& sh, uint32_t ring,
                                             int warp, int lane) {
  using S = TcShape<KV, DP>;
  constexpr int TILE = S::C::TILE, TPW = TILE / kLoadWarps, NW = TPW / 32 ? TPW / 32 : 1;
  constexpr int CPR = S::CPR, RPI = 32 / CPR;  // rows at a time
  auto walk = tree_walk<S::C::ROWS, TILE, S::C::END>(A, sh.start);
  auto at = walk;
  bool bad_page = false, ok = true, more = walk.next(A, at);
  uint32_t n = 0;  // tiles asked for
  int slot = 0;
  const int row0 = lane / CPR, chunk = lane % CPR;  // of this lane, of the first rows
  const bool real_chunk = chunk * 16 < A.dim * S::ES;

  // this lane's tokens (one of every 32 that the warp loads): their pages, asked for a
  // tile ahead
  struct Want {
    int row[NW], page[NW];  // row in the page, -1: none
  };
  auto want = [&](const TcWalk<DP>& p, int t) {
    Want w;
#pragma unroll
    for (int i = 0; i < NW; ++i) {
      const int in = 32 * i + lane, pos = p.s.first + t * TILE + warp * TPW + in;
      w.row[i] = -1;
      w.page[i] = 0;
      if (in < TPW && pos < p.s.len) {
        const int col = A.page_shift >= 0 ? pos >> A.page_shift : pos / A.page;
        w.row[i] = pos - col * A.page;
        w.page[i] = __ldg(A.table + p.b * A.table_stride + col);
      }
    }
    return w;
  };
  struct Place {
    long long off[NW];  // of this lane's tokens in the cache
    uint32_t mask[NW];  // which of the warp's tokens are there
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
    for (int j = 0; j < TPW / RPI; ++j) {
      const int r = j * RPI + row0;
      const long long o = __shfl_sync(0xffffffffu, p.off[j * RPI / 32], r & 31);
      const bool real = (p.mask[j * RPI / 32] >> (r & 31) & 1u) && real_chunk;
      tc_cp16(base + tc_land<KV, DP>(warp * TPW + r, chunk), real ? from + o : A.k, real);
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
    const int kvh = at.x / (at.units / A.heads);
    const bool late = !tc_pair<DP>(A, at);
    auto after = at;
    bool goes_on = true;
    Place now = {}, before = {};
    for (int t = at.t0; ok && t < at.t1 + late; ++t) {
      before = now;
      if (t < at.t1) {
#pragma unroll
        for (int i = 0; i < NW; ++i) {
          const bool in = next.page[i] >= 0 && next.page[i] < A.num_pages;
          const bool live = next.row[i] >= 0 && in;
          bad_page |= next.row[i] >= 0 && !in;
          now.off[i] = live ? next.page[i] * A.s_page + next.row[i] * A.s_token + kvh * A.s_head : 0;
          now.mask[i] = __ballot_sync(0xffffffffu, live);
          if (lane < (TPW < 32 ? TPW / 8 : 4))
            sh.live[slot][warp * (TPW / 8) + 4 * i + lane] =
                static_cast<uint8_t>(now.mask[i] >> (8 * lane));
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
      if (ok && !(late && t == at.t0)) ok = ask(true, late ? before : now);
    }
    at = after;
    more = goes_on;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  if (bad_page && A.err) atomicOr(A.err, MOE_DEVERR_BAD_PAGE);
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
  constexpr int TILE = S::C::TILE, TPW = TILE / kReadyWarps;
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
    uint32_t wild_rows = 0;
    // tokens that are not there: whatever lies in their rows must not count as values
    uint32_t there = 0;
    if (kv) {
      const volatile uint8_t* const live = sh.live[slot] + warp * (TPW / 8);
#pragma unroll
      for (int i = 0; i < TPW / 8; ++i) there |= static_cast<uint32_t>(live[i]) << (8 * i);
    }
    const bool gaps = kv && there != (TPW == 32 ? ~0u : (1u << TPW % 32) - 1);
    const bool care = tame || gaps;
    if constexpr (KV == MOE_KV_E4M3) {
      uint4 raw[TPW / RPI];
#pragma unroll
      for (int j = 0; j < TPW / RPI; ++j)
        raw[j] = tc_lds4(base + tc_land<KV, DP>(warp * TPW + j * RPI + row0, chunk));
      __syncwarp();  // the codes lie where the warp's rows are written
      if (!care) {
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
#pragma unroll
      for (int j = 0; j < TPW / RPI; ++j) {
        if (!care) break;
        const int r = warp * TPW + j * RPI + row0;
        uint4 lo, hi;
        tc_widen(raw[j].x, lo.x, lo.y);
        tc_widen(raw[j].y, lo.z, lo.w);
        tc_widen(raw[j].z, hi.x, hi.y);
        tc_widen(raw[j].w, hi.z, hi.w);
        if (gaps && !(there >> (j * RPI + row0) & 1u)) lo = hi = make_uint4(0, 0, 0, 0);
        if (tame) {
          bool wild = false;
          uint32_t* const w[2] = {&lo.x, &hi.x};
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < 4; ++e) w[h][e] = tc_tame<0x7c00u>(w[h][e], wild);
          if (wild) wild_rows |= 1u << (j * RPI + row0);
        }
        tc_sts4(base + tc_chunk(r, 2 * chunk, S::PANEL), lo);
        tc_sts4(base + tc_chunk(r, 2 * chunk + 1, S::PANEL), hi);
      }
    } else if (care) {
#pragma unroll
      for (int j = 0; j < TPW / RPI; ++j) {
        const uint32_t to = base + tc_chunk(warp * TPW + j * RPI + row0, chunk, S::PANEL);
        if (!(there >> (j * RPI + row0) & 1u)) {
          tc_sts4(to, make_uint4(0, 0, 0, 0));
          continue;
        }
        if (!tame) continue;
        uint4 v = tc_lds4(to);
        bool wild = false;
        v.x = tc_tame<0x7f80u>(v.x, wild);
        v.y = tc_tame<0x7f80u>(v.y, wild);
        v.z = tc_tame<0x7f80u>(v.z, wild);
        v.w = tc_tame<0x7f80u>(v.w, wild);
        if (wild) {
          wild_rows |= 1u << (j * RPI + row0);
          tc_sts4(to, v);
        }
      }
    }
    if (tame) {
      wild_rows = __reduce_or_sync(0xffffffffu, wild_rows);
      if (lane < TPW / 8)
        sh.wild[slot][warp * (TPW / 8) + lane] = static_cast<uint8_t>(wild_rows >> (8 * lane));
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
    const bool late = !tc_pair<DP>(A, at);
    for (int t = at.t0; t < at.t1 + late; ++t) {
      if (t < at.t1 && !ready(false, t)) return;
      if (!(late && t == at.t0) && !ready(true, late ? t - 1 : t)) return;
    }
  }
}

// ------------------------------------------------------------ products (one thread)
template <int KV, int DP>
__device__ __forceinline__ void tc_mma_role(const TreeArgs& A, TcShared& sh, uint32_t qs,
                                            uint32_t ring) {
  using S = TcShape<KV, DP>;
  constexpr int TILE = S::C::TILE, LANES = S::C::LANES, NB = S::NB;
  constexpr uint32_t kS = idesc_make(S::FMT, 128, TILE);
  constexpr uint32_t kO = idesc_make(S::FMT, 128, DP) | (1u << 16);  // V: columns contiguous
  auto walk = tree_walk<S::C::ROWS, TILE, S::C::END>(A, sh.start);
  auto at = walk;
  const uint32_t tmem = sh.tmem;
  long long base = 0;           // tiles of the parts before
  uint32_t q_n[2] = {0, 0};     // phases waited for
  long long seq[2] = {0, 0};    // tiles of a lane before this part
  bool ok = true;
  auto wait = [&](uint64_t* bar, long long phase) {
    ok = ok && mbar_wait(smem_u32(bar), static_cast<uint32_t>(phase) & 1, kTreeWaitNs, &sh.abort);
    return ok;
  };
  while (walk.next(A, at)) {
    const int n = at.t1 - at.t0;
    const bool pair = tc_pair<DP>(A, at);
    for (int l = 0; l <= static_cast<int>(pair); ++l)
      if (!wait(&sh.q_full[l], q_n[l]++)) goto out;
    {
      // the tile that lane l's i-th is, in the part, and the tiles' places in the ring
      auto tile = [&](int l, int i) { return LANES == 1 || pair ? i : 2 * i + l; };
      auto keys = [&](int t) { return base + (pair ? 2ll * t : t == 0 ? 0 : 2ll * t - 1); };
      auto vals = [&](int t) { return base + (pair || t == n - 1 ? 2ll * t + 1 : 2ll * t + 2); };
      auto issue_s = [&](int l, int i) {
        const int t = tile(l, i);
        const long long k = keys(t), q = seq[l] + i;
        const int buf = static_cast<int>(k % S::RING), b = NB == 2 ? static_cast<int>(q & 1) : l;
        if (!wait(&sh.full[buf], k / S::RING)) return;
        // the S tile holds the weights of the lane's tile NB before: used up
        if (q >= NB && !wait(&sh.o_full[b], NB == 2 ? q / 2 - 1 : q - 1)) return;
        tc_fence_after();
        const uint32_t qa = qs + (pair ? l : 0) * S::QBLOCK, ka = ring + buf * S::BUF;
#pragma unroll
        for (int ks = 0; ks < DP / 16; ++ks)
          mma_issue<1>(tmem + b * TILE, sdesc_sw128(qa + ks / 4 * 16384 + ks % 4 * 32),
                       sdesc_sw128(ka + ks / 4 * S::PANEL + ks % 4 * 32), kS, ks > 0);
        mma_commit(smem_u32(&sh.s_full[b]));
        if (!pair || l == 1) mma_commit(smem_u32(&sh.empty[buf]));
      };
      auto issue_o = [&](int l, int i) {
        const int t = tile(l, i);
        const long long v = vals(t), q = seq[l] + i;
        const int buf = static_cast<int>(v % S::RING), b = NB == 2 ? static_cast<int>(q & 1) : l;
        if (!wait(&sh.p_full[b], NB == 2 ? q / 2 : q)) return;
        if (!wait(&sh.full[buf], v / S::RING)) return;
        tc_fence_after();
        const uint32_t va = ring + buf * S::BUF;
#pragma unroll
        for (int ks = 0; ks < TILE / 16; ++ks)
          tc_mma_ts(tmem + 256 + l * DP, tmem + b * TILE + 8 * ks,
                    tc_desc_tokens(va + ks * 2048, S::PANEL), kO, i > 0 || ks > 0);
        mma_commit(smem_u32(&sh.o_full[b]));
        if (!pair || l == 1) mma_commit(smem_u32(&sh.empty[buf]));
      };
      const int n0 = LANES == 1 || pair ? n : (n + 1) / 2, n1 = LANES == 1 ? 0 : pair ? n : n / 2;
      issue_s(0, 0);
      if (ok && n1 > 0) issue_s(1, 0);
      for (int i = 0; ok && i < n0; ++i) {
        if (NB == 2 && i + 1 < n0) issue_s(0, i + 1);
        if (ok) issue_o(0, i);
        if (ok && NB == 1 && i + 1 < n0) issue_s(0, i + 1);
        if (ok && i < n1) issue_o(1, i);
        if (ok && i + 1 < n1) issue_s(1, i + 1);
      }
      seq[0] += n0;
      seq[1] += n1;
      base += 2ll * n;
    }
  }
out:
  if (!ok) {
    atomicExch(&sh.abort, 1);
    // nothing of this CTA's may be under way when its memory goes
    mma_commit(smem_u32(&sh.drain));
    int never = 0;
    mbar_wait(smem_u32(&sh.drain), 0, kTreeWaitNs, &never);
  }
}

// ------------------------------------------------------------ softmax
template <int KV, int DP>
__device__ __forceinline__ void tc_softmax_role(const TreeArgs& A, TcShared& sh, TcTurns& turns,
                                                uint32_t qs, int warp, int lane) {
  using S = TcShape<KV, DP>;
  constexpr int TILE = S::C::TILE, LANES = S::C::LANES, NB = S::NB, CH = TILE / 32;
  const int l = warp >> 2, r = (warp & 3) * 32 + lane;  // lane of the CTA, row of its block
  if (l >= LANES) return;
  auto walk = tree_walk<S::C::ROWS, TILE, S::C::END>(A, sh.start);
  auto at = walk;
  const uint32_t tmem = sh.tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
  const uint32_t t_o = tmem + 256 + l * DP;
  long long seq = 0, tiles = 0, joins = 0;
  bool ok = true;
  auto wait = [&](uint64_t* bar, long long phase) {
    ok = mbar_wait(smem_u32(bar), static_cast<uint32_t>(phase) & 1, kTreeWaitNs, &sh.abort);
    return __all_sync(0xffffffffu, ok);
  };
  // the product with the weights of the lane's tile q.  (A barrier tells a phase
  // from the one before it only, and with two S tiles two products may be under
  // way: a barrier for each)
  auto wait_o = [&](long long q) -> bool {
    return NB == 2 ? wait(&sh.o_full[q & 1], q / 2) : wait(&sh.o_full[l], q);
  };
  while (walk.next(A, at)) {
    const TreeSpan& s = at.s;
    const int blocks = at.units / A.heads;
    const int kvh = at.x / blocks, r0 = at.x % blocks * S::C::ROWS;
    const int rows = min(S::C::ROWS, s.use * A.group - r0);
    const bool pair = tc_pair<DP>(A, at), alternate = LANES == 2 && !pair;
    const int R = r0 + (pair ? 128 * l : 0) + r;
    const bool mine = R < r0 + rows;
    const int Rc = min(R, r0 + rows - 1), node = Rc / A.group, h = kvh * A.group + Rc - node * A.group;
    const long long row = s.row0 + node;
    // a warp whose rows are all beyond the block's only keeps step
    const bool idle = (pair ? 128 * l : 0) + (warp & 3) * 32 >= rows;
    const TreeMask mask = tree_mask(A, s, node);
    float sl = A.scale_log2, v_mul = 1.0f, f = 0.0f;  // f: of logits, in base 2
    if constexpr (KV == MOE_KV_E4M3) {
      sl *= A.k_scale[kvh];
      v_mul = A.v_scale[kvh];
    }
    // ---- the block's row of Q; a negative scale turns its sign instead of the
    // logits', so that the largest product is the largest logit
    if (l == 0 || pair) {
      const uint32_t to = qs + (pair ? l : 0) * S::QBLOCK;
      const uint32_t sign = sl < 0.0f ? 0x80008000u : 0u;
      const uint4* const q = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(A.q) +
                                                            row * A.q_n + h * A.q_h);
      constexpr int HALF = DP / 8 < 16 ? DP / 8 : 16;  // chunks at a time
      float mul = 1.0f, inv = 1.0f;
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
        if (alternate) turns.q_mul[r] = mul;
      }
#pragma unroll
      for (int c0 = 0; c0 < DP / 8; c0 += HALF) {
        uint4 v[HALF];
#pragma unroll
        for (int c = 0; c < HALF; ++c) {
          v[c] = make_uint4(0, 0, 0, 0);
          if (mine && (c0 + c) * 8 < A.dim) v[c] = __ldg(q + c0 + c);
        }
#pragma unroll
        for (int c = 0; c < HALF; ++c) {
          v[c].x ^= sign;
          v[c].y ^= sign;
          v[c].z ^= sign;
          v[c].w ^= sign;
          if constexpr (KV == MOE_KV_E4M3) {
            uint32_t* const w = &v[c].x;
#pragma unroll
            for (int e = 0; e < 4; ++e)
              w[e] = tc_f16x2(__uint_as_float(w[e] << 16) * inv,
                              __uint_as_float(w[e] & 0xffff0000u) * inv);
          }
          tc_sts4(to + tc_chunk(r, c0 + c, 16384), v[c]);
        }
      }
      fence_proxy_async_shared();
      mbar_arrive(smem_u32(&sh.q_full[l]));
      f = fmaxf(fabsf(sl) * mul, kTcLeast);
    }
    const int n = at.t1 - at.t0;
    const int mine_n = alternate ? (n + 1 - l) / 2 : n;
    const int low = tree_low(A, s, mask);
    float m = -INFINITY, sum = 0.0f;
    for (int i = 0; i < mine_n; ++i) {
      const int t = alternate ? 2 * i + l : i;
      const int pos = s.first + (at.t0 + t) * TILE;
      const long long q = seq + i;
      const int b = NB == 2 ? static_cast<int>(q & 1) : l;
      const uint32_t t_s = tmem + b * TILE;
      if (!wait(&sh.s_full[b], NB == 2 ? q / 2 : q)) goto out;
      if (idle) {
        mbar_arrive(smem_u32(&sh.p_full[b]));
        continue;
      }
      tc_fence_after();
      if (i == 0 && alternate && l == 1) {
        f = fmaxf(fabsf(sl) * (KV == MOE_KV_E4M3 ? turns.q_mul[r] : 1.0f), kTcLeast);
      }
      const int slot = static_cast<int>((tiles + t) % kSlots);
      // (loops over the columns are rolled up: a longer program, most of it run once
      // a tile, was fetched for 6 us at the first tile that masks apply to)
      auto attended = [&](int c) {
        return *reinterpret_cast<const volatile uint32_t*>(&sh.live[slot][4 * c]) &
               tree_attends(s, mask, low, pos + 32 * c);
      };
      const bool masked = tc_masked<TILE>(A, s, pos);
      bool all = !masked, any = true;
#pragma unroll
      for (int c = 0; c < CH; ++c)
        all = all && *reinterpret_cast<const volatile uint32_t*>(&sh.live[slot][4 * c]) == ~0u;
      float top = -INFINITY;
      auto largest = [&](const float (&v)[32]) {
        float x[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
        for (int j = 4; j < 32; ++j) x[j & 3] = fmaxf(x[j & 3], v[j]);
        top = fmaxf(top, fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])));
      };
      if (all) {  // (the same for all rows)
#pragma unroll 1
        for (int c = 0; c < CH; ++c) {
          float v[32];
          tmem_ld32(t_s + 32 * c, v);
          tmem_wait_ld(v);
          largest(v);
        }
      } else {  // logits that do not count become -inf
        any = false;
#pragma unroll 1
        for (int c = 0; c < CH; ++c) {
          float v[32];
          tmem_ld32(t_s + 32 * c, v);
          const uint32_t word = attended(c);
          any = any || word;
          tmem_wait_ld(v);
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = word >> j & 1u ? v[j] : -INFINITY;
          largest(v);
          tc_st32(t_s + 32 * c, v);
        }
        tc_wait_st();
      }
      top = top == -INFINITY ? top : top * f;
      const bool grow = top > m + (S::LIFT + S::LAG);
      float keep = 1.0f;
      if (grow) {
        const float to = top - S::LIFT;
        keep = tree_ex2(m - to);
        m = to;
        sum *= keep;
      }
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
      // from here on the row has tokens, if only of logits -inf: m says so
      if (any) m = fmaxf(m, -FLT_MAX);
      const float ref = m == -INFINITY ? 0.0f : m;
      float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
      for (int c = 0; c < CH; ++c) {
        float v[32];
        tmem_ld32(t_s + 32 * c, v);
        tmem_wait_ld(v);
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = tree_ex2(fmaf(v[j], f, -ref));
        uint32_t p[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          part[j & 3] += v[2 * j] + v[2 * j + 1];
          p[j] = KV == MOE_KV_E4M3 ? tc_f16x2(v[2 * j], v[2 * j + 1])
                                   : tree_bf16x2(v[2 * j], v[2 * j + 1]);
        }
        tc_st16(t_s + 16 * c, p);
      }
      sum += (part[0] + part[1]) + (part[2] + part[3]);
      tc_wait_st();
      tc_fence_before();
      mbar_arrive(smem_u32(&sh.p_full[b]));
      if (masked) {
        // values that are not finite: what they leave in the rows that attend them
        // (told before the values' barrier, which this product has waited for)
        if (!wait_o(q)) goto out;
        tc_fence_after();
        uint32_t wild = 0;
#pragma unroll
        for (int c = 0; c < CH; ++c)
          wild |= *reinterpret_cast<const volatile uint32_t*>(&sh.wild[slot][4 * c]);
        if (wild) {
#pragma unroll 1
          for (int d0 = 0; d0 < DP; d0 += 32) {
            float o[32];
            tmem_ld32(t_o + d0, o);
            tmem_wait_ld(o);
#pragma unroll 1
            for (int c = 0; c < CH; ++c) {
              uint32_t left =
                  *reinterpret_cast<const volatile uint32_t*>(&sh.wild[slot][4 * c]) & attended(c);
              while (left) {
                const int tok = pos + 32 * c + __ffs(left) - 1;
                left &= left - 1;
                const int col = A.page_shift >= 0 ? tok >> A.page_shift : tok / A.page;
                const char* const v = A.v + A.table[at.b * A.table_stride + col] * A.s_page +
                                      (tok - col * A.page) * A.s_token + kvh * A.s_head;
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                  if (d0 + j >= A.dim) continue;
                  float x;
                  if constexpr (KV == MOE_KV_E4M3) {
                    const uint8_t e = *reinterpret_cast<const uint8_t*>(v + d0 + j);
                    x = (e & 0x7f) == 0x7f ? __uint_as_float(0x7fffffffu) : 0.0f;
                  } else {
                    x = __uint_as_float(
                        static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(v + 2 * (d0 + j)))
                        << 16);
                    if (fabsf(x) <= FLT_MAX) x = 0.0f;
                  }
                  o[j] += x;
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
    seq += mine_n;
    tiles += n;
    if (mine_n > 0) {
      if (!wait_o(seq - 1)) goto out;
      tc_fence_after();
    }
    // ---- the part's end: the lanes that took turns join, each half of the columns
    {
      float k[2] = {1.0f, 0.0f}, top = m, total = sum;
      if (alternate) {
        turns.m[l][r] = m;
        turns.sum[l][r] = sum;
        tc_fence_before();
        mbar_arrive(smem_u32(&sh.join[0]));
        if (!wait(&sh.join[0], joins)) goto out;
        tc_fence_after();
        const float m0 = turns.m[0][r], m1 = turns.m[1][r];
        top = fmaxf(m0, m1);
        k[0] = top == -INFINITY ? 1.0f : tree_ex2(m0 - top);
        k[1] = top == -INFINITY ? 1.0f : tree_ex2(m1 - top);
        total = k[0] * turns.sum[0][r] + k[1] * turns.sum[1][r];
      }
      const bool two = alternate && n > 1;
      const bool whole = at.t0 == 0 && at.t1 == at.nt;
      const float inv = top == -INFINITY ? 0.0f : v_mul / total;
      const long long part = 2ll * blockIdx.x + (at.t0 == 0 ? 0 : 1);
      const int prow = (pair ? 128 * l : 0) + r;
      const uint32_t o_base = tmem + 256 + (pair ? l * DP : 0);
      constexpr int W = 32;
#pragma unroll 1
      for (int d = alternate ? l * (DP / 2) : 0;
           !idle && d < (alternate ? (l + 1) * (DP / 2) : DP); d += W) {
        float o[W];
        tmem_ld32(o_base + d, o);
        tmem_wait_ld(o);
        if (alternate) {
          if (two) {
            float u[W];
            tmem_ld32(o_base + DP + d, u);
            tmem_wait_ld(u);
#pragma unroll
            for (int j = 0; j < W; ++j) o[j] = k[0] * o[j] + k[1] * u[j];
          } else {
#pragma unroll
            for (int j = 0; j < W; ++j) o[j] *= k[0];
          }
        }
        if (!mine) continue;
        if (whole) {
#pragma unroll
          for (int j = 0; j < W; j += 8)
            if (d + j < A.dim)
              *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(A.out) + row * A.o_n +
                                        h * A.o_h + d + j) =
                  make_uint4(tree_bf16x2(o[j] * inv, o[j + 1] * inv),
                             tree_bf16x2(o[j + 2] * inv, o[j + 3] * inv),
                             tree_bf16x2(o[j + 4] * inv, o[j + 5] * inv),
                             tree_bf16x2(o[j + 6] * inv, o[j + 7] * inv));
        } else {
#pragma unroll
          for (int j = 0; j < W; j += 4)
            *reinterpret_cast<float4*>(A.part_o + (part * S::C::ROWS + prow) * DP + d + j) =
                make_float4(o[j], o[j + 1], o[j + 2], o[j + 3]);
        }
      }
      if (mine && (l == 0 || pair)) {
        if (!whole) A.part_ml[part * S::C::ROWS + prow] = make_float2(top, total);
        else if (A.lse) A.lse[row * A.Hq + h] = tree_lse<KV>(top, total);
      }
      if (l == 0 && r == 0 && at.t1 < at.nt) tree_record(A, sh.start, at);
      tc_fence_before();
      if (alternate) {  // neither's accumulator is written while the other reads it
        mbar_arrive(smem_u32(&sh.join[1]));
        if (!wait(&sh.join[1], joins)) goto out;
        ++joins;
      }
    }
  }
out:
  if (!ok) {
    atomicExch(&sh.abort, 1);
    if (A.err) atomicOr(A.err, MOE_DEVERR_TIMEOUT);
  }
}

template <int KV, int DP>
__global__ void __launch_bounds__(kTcThreads, 1)
    tree_tc_kernel(const TreeArgs A, const __grid_constant__ CUtensorMap k_map,
                   const __grid_constant__ CUtensorMap v_map) {
  using S = TcShape<KV, DP>;
  extern __shared__ uint8_t tc_smem[];
  const uint32_t base = (smem_u32(tc_smem) + 1023) & ~1023u;
  const uint32_t qs = base, ring = base + S::C::LANES * S::QBLOCK;
  uint8_t* const behind_q = tc_smem + (ring - smem_u32(tc_smem));
  TcShared& sh = *reinterpret_cast<TcShared*>(behind_q + S::RING * S::BUF);
  TcTurns& turns = *reinterpret_cast<TcTurns*>(behind_q - S::QBLOCK);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_wait();
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(&sh.tmem), 512);
    tmem_relinquish();
  }
  if (tid == 0) {
    for (int i = 0; i < S::RING; ++i) {
      mbar_init(smem_u32(&sh.landed[i]), A.box ? 1 : 33 * kLoadWarps);
      mbar_init(smem_u32(&sh.full[i]), kReadyWarps);
      mbar_init(smem_u32(&sh.empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&sh.s_full[i]), 1);
      mbar_init(smem_u32(&sh.p_full[i]), 128);
      mbar_init(smem_u32(&sh.o_full[i]), 1);
      mbar_init(smem_u32(&sh.q_full[i]), 128);
      mbar_init(smem_u32(&sh.join[i]), 256);
    }
    mbar_init(smem_u32(&sh.drain), 1);
    fence_mbar_init();
    sh.abort = 0;
  }
  tc_fence_before();
  pdl_trigger();
  tree_begin<S::C::ROWS, S::C::TILE, S::C::END>(A, &sh.start, sh.sums);
  tc_fence_after();
  if (warp < 8) {
    tc_softmax_role<KV, DP>(A, sh, turns, qs, warp, lane);
  } else if (warp < 8 + kLoadWarps) {
    if (A.box == 0) tc_load_role<KV, DP>(A, sh, ring, warp - 8, lane);
    else if (warp == 8) tc_tma_role<KV, DP>(A, &k_map, &v_map, sh, ring, lane);
  } else if (warp < kMmaWarp) {
    tc_ready_role<KV, DP>(A, sh, ring, warp - 8 - kLoadWarps, lane);
  } else if (lane == 0) {
    tc_mma_role<KV, DP>(A, sh, qs, ring);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(sh.tmem, 512);
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
  constexpr int SMEM = 1024 + S::C::LANES * S::QBLOCK + S::RING * S::BUF + kTcShared;
  static_assert(SMEM <= 227 * 1024, "shared memory of an SM");
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
