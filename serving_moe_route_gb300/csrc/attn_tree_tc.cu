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
//   loads    four warps fill a ring of key and value tiles with 16-byte
//            cp.async, LOOK tiles ahead, across unit borders; any page size and
//            strides.  e4m3 codes land in the half of their tile that the same
//            warp will write, and are widened to f16, which holds them exactly,
//            on the way to the full barrier.
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
constexpr int kLoadWarps = 4, kMmaWarp = 8 + kLoadWarps;
static_assert(kTcThreads == 32 * (kMmaWarp + 1), "two softmax warpgroups, loads, products");

template <int KV, int DP>
struct TcShape {
  using C = TcCfg<DP>;
  static constexpr int RING = 163840 / (C::TILE * DP * 2);
  static constexpr int LOOK = RING - 2;            // tiles on their way
  static constexpr int BUF = C::TILE * DP * 2;     // bytes of a tile
  static constexpr int PANEL = C::TILE * 128;      // of 64 columns of it
  static constexpr int QBLOCK = 128 * DP * 2;
  static constexpr int NB = C::LANES == 1 ? 2 : 1; // S tiles of a lane
  static constexpr int ES = kv_esize(KV);
  static constexpr int CPR = DP * ES / 16;         // 16-byte chunks of a cached row
  static constexpr int TPW = C::TILE / kLoadWarps; // tokens of a tile that a warp loads
  static constexpr int RPI = 32 / CPR;             // of them at a time
  static constexpr float LIFT = KV == MOE_KV_E4M3 ? kTreeLift : 0.0f;
  static constexpr float LAG = KV == MOE_KV_E4M3 ? 2.0f : 8.0f;
  static constexpr uint32_t FMT = KV == MOE_KV_E4M3 ? 0 : 1;  // f16, bf16
};
constexpr int kSlots = 8;  // tiles whose live and non-finite tokens are kept

// The second block of Q's memory where a unit has one block only: what the
// lanes that take turns tell each other
struct TcTurns {
  float m[2][128], sum[2][128], q_mul[128];
};
// What lies behind the tiles in shared memory
struct TcShared {
  uint64_t full[10], empty[10], s_full[2], p_full[2], o_full[2], q_full[2], join[2], drain;
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
template <int KV, int DP>
__device__ __forceinline__ void tc_load_role(const TreeArgs& A, TcShared& sh, uint32_t ring,
                                             int warp, int lane) {
  using S = TcShape<KV, DP>;
  constexpr int TILE = S::C::TILE, TPW = S::TPW, CPR = S::CPR, RPI = S::RPI;
  auto walk = tree_walk<S::C::ROWS, TILE, S::C::END>(A, sh.start);
  auto at = walk;
  bool bad_page = false, more = walk.next(A, at);
  long long n = 0;  // tiles asked for
  uint32_t masked = 0;  // bit i: tile n - 1 - i is one of values that masks apply to
  const int row0 = lane / CPR, chunk = lane % CPR;  // of this lane, of the first rows
  const bool real_chunk = chunk * 16 < A.dim * S::ES;

  // the last step of tile i: what cp.async has brought is made ready and told
  auto ready = [&](long long i, bool tame) {
    const int buf = static_cast<int>(i % S::RING);
    const uint32_t base = ring + buf * S::BUF;
    uint32_t wild_rows = 0;
    if constexpr (KV == MOE_KV_E4M3) {
      uint4 raw[TPW / RPI];
#pragma unroll
      for (int j = 0; j < TPW / RPI; ++j)
        raw[j] = tc_lds4(base + tc_chunk(warp * TPW + j * RPI + row0, CPR + chunk, S::PANEL));
      __syncwarp();  // the codes lie where the warp's rows are written
#pragma unroll
      for (int j = 0; j < TPW / RPI; ++j) {
        const int r = warp * TPW + j * RPI + row0;
        uint4 lo, hi;
        tc_widen(raw[j].x, lo.x, lo.y);
        tc_widen(raw[j].y, lo.z, lo.w);
        tc_widen(raw[j].z, hi.x, hi.y);
        tc_widen(raw[j].w, hi.z, hi.w);
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
    } else if (tame) {
#pragma unroll
      for (int j = 0; j < TPW / RPI; ++j) {
        const uint32_t to = base + tc_chunk(warp * TPW + j * RPI + row0, chunk, S::PANEL);
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
        sh.wild[(i / 2) % kSlots][warp * (TPW / 8) + lane] =
            static_cast<uint8_t>(wild_rows >> (8 * lane));
    }
    fence_proxy_async_shared();
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&sh.full[buf]));
  };

  // this lane's token (the first TPW lanes have one): its page, asked for a tile ahead
  struct Want {
    int row, page;  // row in the page, -1: none
  };
  auto want = [&](const TcWalk<DP>& p, int t) {
    Want w = {-1, 0};
    const int pos = p.s.first + t * TILE + warp * TPW + lane;
    if (lane < TPW && pos < p.s.len) {
      const int col = A.page_shift >= 0 ? pos >> A.page_shift : pos / A.page;
      w.row = pos - col * A.page;
      w.page = __ldg(A.table + p.b * A.table_stride + col);
    }
    return w;
  };
  Want next = {-1, 0};
  if (more) next = want(at, at.t0);
  while (more) {
    const int kvh = at.x / (at.units / A.heads);
    auto after = at;
    bool goes_on = true;
    for (int t = at.t0; t < at.t1; ++t) {
      const bool in = next.page >= 0 && next.page < A.num_pages;
      const bool live = next.row >= 0 && in;
      bad_page |= next.row >= 0 && !in;
      const long long off =
          live ? next.page * A.s_page + next.row * A.s_token + kvh * A.s_head : 0;
      const uint32_t mask = __ballot_sync(0xffffffffu, live);
      if (t + 1 < at.t1) {
        next = want(at, t + 1);
      } else {
        goes_on = walk.next(A, after);
        if (goes_on) next = want(after, after.t0);
      }
      if (lane < TPW / 8)
        sh.live[(n / 2) % kSlots][warp * (TPW / 8) + lane] = static_cast<uint8_t>(mask >> (8 * lane));
#pragma unroll 1
      for (int kv = 0; kv < 2; ++kv) {
        const int buf = static_cast<int>(n % S::RING);
        if (n >= S::RING &&
            !mbar_wait(smem_u32(&sh.empty[buf]), static_cast<uint32_t>(n / S::RING - 1) & 1,
                       kTreeWaitNs, &sh.abort)) {
          atomicExch(&sh.abort, 1);
          asm volatile("cp.async.wait_group 0;" ::: "memory");
          return;
        }
        const uint32_t base = ring + buf * S::BUF;
        const char* const from = (kv ? A.v : A.k) + chunk * 16;
#pragma unroll
        for (int j = 0; j < TPW / RPI; ++j) {
          const int r = j * RPI + row0;
          const long long o = __shfl_sync(0xffffffffu, off, r);
          const bool real = (mask >> r & 1u) && real_chunk;
          tc_cp16(base + tc_chunk(warp * TPW + r, KV == MOE_KV_E4M3 ? CPR + chunk : chunk, S::PANEL),
                  real ? from + o : A.k, real);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        ++n;
        masked = masked << 1 | (kv && tc_masked<TILE>(A, at.s, at.s.first + t * TILE));
        if (n > S::LOOK) {
          asm volatile("cp.async.wait_group %0;" ::"n"(S::LOOK) : "memory");
          ready(n - 1 - S::LOOK, masked >> S::LOOK & 1u);
        }
      }
    }
    at = after;
    more = goes_on;
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  for (long long i = n > S::LOOK ? n - S::LOOK : 0; i < n; ++i) ready(i, masked >> (n - 1 - i) & 1u);
  if (bad_page && A.err) atomicOr(A.err, MOE_DEVERR_BAD_PAGE);
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
    const int blocks = at.units / A.heads;
    const int rows = min(S::C::ROWS, at.s.use * A.group - at.x % blocks * S::C::ROWS);
    const bool pair = LANES == 2 && rows > 128;
    for (int l = 0; l <= static_cast<int>(pair); ++l)
      if (!wait(&sh.q_full[l], q_n[l]++)) goto out;
    {
      // the tile that lane l's i-th is, in the part
      auto tile = [&](int l, int i) { return LANES == 1 || pair ? i : 2 * i + l; };
      auto issue_s = [&](int l, int i) {
        const int t = tile(l, i);
        const long long k = base + 2ll * t, q = seq[l] + i;
        const int buf = static_cast<int>(k % S::RING), b = NB == 2 ? static_cast<int>(q & 1) : l;
        if (!wait(&sh.full[buf], k / S::RING)) return;
        // the S tile holds the weights of the lane's tile NB before: used up
        if (q >= NB && !wait(&sh.o_full[l], q - NB)) return;
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
        const long long v = base + 2ll * t + 1, q = seq[l] + i;
        const int buf = static_cast<int>(v % S::RING), b = NB == 2 ? static_cast<int>(q & 1) : l;
        if (!wait(&sh.p_full[b], NB == 2 ? q / 2 : q)) return;
        if (!wait(&sh.full[buf], v / S::RING)) return;
        tc_fence_after();
        const uint32_t va = ring + buf * S::BUF;
#pragma unroll
        for (int ks = 0; ks < TILE / 16; ++ks)
          tc_mma_ts(tmem + 256 + l * DP, tmem + b * TILE + 8 * ks,
                    tc_desc_tokens(va + ks * 2048, S::PANEL), kO, i > 0 || ks > 0);
        mma_commit(smem_u32(&sh.o_full[l]));
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
  while (walk.next(A, at)) {
    const TreeSpan& s = at.s;
    const int blocks = at.units / A.heads;
    const int kvh = at.x / blocks, r0 = at.x % blocks * S::C::ROWS;
    const int rows = min(S::C::ROWS, s.use * A.group - r0);
    const bool pair = LANES == 2 && rows > 128, alternate = LANES == 2 && !pair;
    const int R = r0 + (pair ? 128 * l : 0) + r;
    const bool mine = R < r0 + rows;
    const int Rc = min(R, r0 + rows - 1), node = Rc / A.group, h = kvh * A.group + Rc - node * A.group;
    const long long row = s.row0 + node;
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
      f = fabsf(sl) * mul;
    }
    const int n = at.t1 - at.t0;
    const int mine_n = alternate ? (n + 1 - l) / 2 : n;
    const int low = tree_low(A, s, node);
    float m = -INFINITY, sum = 0.0f;
    for (int i = 0; i < mine_n; ++i) {
      const int t = alternate ? 2 * i + l : i;
      const int pos = s.first + (at.t0 + t) * TILE;
      const long long q = seq + i;
      const int b = NB == 2 ? static_cast<int>(q & 1) : l;
      const uint32_t t_s = tmem + b * TILE;
      if (!wait(&sh.s_full[b], NB == 2 ? q / 2 : q)) goto out;
      tc_fence_after();
      if (i == 0 && alternate && l == 1) {
        f = fabsf(sl);
        if constexpr (KV == MOE_KV_E4M3) f *= turns.q_mul[r];
      }
      const int slot = static_cast<int>((tiles + t) % kSlots);
      uint32_t word[CH];
      bool all = !tc_masked<TILE>(A, s, pos);
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        word[c] = *reinterpret_cast<const volatile uint32_t*>(&sh.live[slot][4 * c]);
        all = all && word[c] == ~0u;
      }
      bool any = true;
      if (!all) {  // (the same for all rows)
        any = false;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          word[c] &= tree_attends(A, s, node, low, pos + 32 * c);
          any = any || word[c];
        }
      }
      float top = -INFINITY;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        float v[32];
        tmem_ld32(t_s + 32 * c, v);
        tmem_wait_ld(v);
        if (!all) {
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = word[c] >> j & 1u ? v[j] : -INFINITY;
        }
        float x[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
        for (int j = 4; j < 32; ++j) x[j & 3] = fmaxf(x[j & 3], v[j]);
        top = fmaxf(top, fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])));
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
        if (!wait(&sh.o_full[l], q - 1)) goto out;
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
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        float v[32];
        tmem_ld32(t_s + 32 * c, v);
        tmem_wait_ld(v);
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = tree_ex2(fmaf(v[j], f, -ref));
        if (!all) {
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = word[c] >> j & 1u ? v[j] : 0.0f;
        }
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
      if (!all && tc_masked<TILE>(A, s, pos)) {
        // values that are not finite: what they leave in the rows that attend them
        // (told before the values' barrier, which this product has waited for)
        if (!wait(&sh.o_full[l], q)) goto out;
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
                  *reinterpret_cast<const volatile uint32_t*>(&sh.wild[slot][4 * c]) & word[c];
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
      if (!wait(&sh.o_full[l], seq - 1)) goto out;
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
      for (int d = alternate ? l * (DP / 2) : 0; d < (alternate ? (l + 1) * (DP / 2) : DP); d += W) {
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
__global__ void __launch_bounds__(kTcThreads, 1) tree_tc_kernel(const TreeArgs A) {
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
      mbar_init(smem_u32(&sh.full[i]), kLoadWarps);
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
    tc_load_role<KV, DP>(A, sh, ring, warp - 8, lane);
  } else if (lane == 0) {
    tc_mma_role<KV, DP>(A, sh, qs, ring);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(sh.tmem, 512);
}

template <int KV, int DP>
static cudaError_t launch_tc(const TreeArgs& a, int ctas, cudaStream_t st) {
  using S = TcShape<KV, DP>;
  constexpr int SMEM = 1024 + S::C::LANES * S::QBLOCK + S::RING * S::BUF + kTcShared;
  static_assert(SMEM <= 227 * 1024, "shared memory of an SM");
  auto* kern = tree_tc_kernel<KV, DP>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), SMEM, done);
  if (e != cudaSuccess) return e;
  e = launch_chained(kern, dim3(ctas), dim3(kTcThreads), SMEM, st, a);
  if (e != cudaSuccess) return e;
  return launch_chained(tree_join_kernel<KV, DP, S::C::ROWS>, dim3(ctas), dim3(32 * kTreeJoinWarps),
                        0, st, a);
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
