// attn_decode.cu -- attention of one new token per request over the paged
// key-value cache (moe_attn_decode, include/moe_route.h).
//
// With G = Hq / kv_heads query heads on each cached head, every cached
// element is used by 2G flops and read once: for the G of real models (1 to
// 16) the operator is bound by the cache's bytes, so the kernel is built to
// keep loads in flight, and the products only have to keep out of the way.
//
//   work     A unit is (request, kv head, block of 16 query heads); its tokens
//            form tiles, a stage per warp, and it counts its tiles and one or
//            two more for its end, which takes as long.  The counts of all
//            units, in order, are cut into equal contiguous ranges, one per CTA
//            of a single wave, so ragged lengths and long single requests
//            balance alike; a range may begin and end inside a unit.
//   loads    Each warp has a ring of ST stages of 8 to 32 keys and values and
//            fills it with 16-byte cp.async, ST-1 stages ahead, across unit
//            borders; page ids are fetched one stage before that.  Warps
//            share nothing in the loop: no CTA-wide barrier, no producer.
//            Rows that follow one another in one page (every stage of pages of
//            16 tokens or more, but for windows) need no address of their own.
//   math     S = Q K^T and O += P V on m16n8k16 (bf16; e4m3 as f16, which holds
//            it exactly) and m16n8k8 (f32 as two 11-bit terms) tensor core
//            instructions with the 16 query heads as rows.  One pass keeps a
//            reference m and the sum l of each row in fp32 (base 2); m is a
//            logit that was the largest when it was taken, and O is rescaled
//            only when one lies 8 above it, so that weights stay below 2^8
//            (e4m3's, which are f16: below 2^15, LIFT and LAG below).  tcgen05
//            needs 128 rows on its M side and its result in tensor memory; here
//            one operand has 16 rows or fewer and the softmax works on its rows
//            between the two products.  The m16n8 instructions suffice: without
//            the loads' waiting a bf16 tile takes a third of the time of its
//            bytes.  e4m3 products of e4m3 operands (m16n8k32) were tried: 1.8
//            times as long as f16's, and sums 2^-8 off.
//   joining  At a unit's end the CTA's warps join through shared memory.  A
//            unit inside one range is written at once; parts of a unit cut by
//            range borders go to the workspace in fp32 and the second kernel
//            joins them in range order: no atomics, one fixed result.
//
// Bound by the cache's bytes on long lengths and by a fixed part otherwise, 7
// us: 4 before the first product (lengths, page ids, first rows) and 1 to 2 for
// the second kernel, which is left out where no unit can be cut.  Measured on a
// GB300, 32 query heads on 4 of 128: one request of 262161 tokens, bf16: 87 us,
// 6.1 TB/s (91% of the copy bandwidth); 256 up to 8192, e4m3: 128 us, 5.7 TB/s;
// 64 up to 4096, bf16: 36 us, 4.8 TB/s, f32: 88 us, 3.9 TB/s, whose split
// operands' instructions bound it; one of 700: 7 us.
//
// Where fewer bits than fp32 are held: weights are a pair of bf16 (2^-16) or of
// tf32 terms, or f16 (e4m3 caches, 2^-11); f32 operands are pairs of tf32 terms;
// and O of bf16 and e4m3 caches is summed in the instructions' accumulator, fp32
// but cut: 2^-23 of it an instruction, 2^-10 at most for a warp's 2^16 tokens.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cfloat>
#include <climits>
#include <cmath>
#include <cstdint>

#include "../../include/moe_route.h"
#include "decode_internal.cuh"
#include "moe_internal.cuh"
#include "ptx.cuh"

namespace moe {

constexpr int kRows = 16;  // query heads of a unit: the m of the mma instructions
constexpr int kMaxLen = INT_MAX - 1024;  // a tile's end stays an int

struct AttnArgs {
  const char *k, *v;
  long long s_page, s_token, s_head;  // bytes
  const float *k_scale, *v_scale;
  const void* q;
  long long q_b, q_h;  // elements
  void* out;
  long long o_b, o_h;  // elements
  float* lse;
  const int* table;
  long long table_stride;
  const int* lens;
  float* part_o;   // [2 * ctas][16][DP]
  float2* part_ml; // [2 * ctas][16]
  int4* info;      // [ctas] {unit's request, unit in request, parts, 0}
  unsigned* err;
  float scale_log2;
  int B, Hq, heads, group, blocks;  // blocks: of 16 query heads per kv head
  int dim, page, page_shift, num_pages, max_pages, window;
};

// ------------------------------------------------------------ instructions
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool real) {
  // a row that is not real is filled with zeros and nothing is read
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(real ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint4 lds4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ uint2 lds2(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_tf32(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// x = hi + lo: hi is x rounded to 11 bits, lo has the 12 bits (and a sign) that
// are left, of which the instruction cuts the last where there are so many:
// 2^-23 of x.  Products of two such pairs without lo * lo are off by 2^-21 of
// |x y| at most (and by 2^-136 of each factor: subnormal terms' last places).
// hi stays finite: a NaN is one in lo, and an infinity is lo's, so that a
// logit, or a value by its weight, is the infinity that it is without a split.
__device__ __forceinline__ void split_tf32(float x, uint32_t& hi, uint32_t& lo) {
  float y;  // with x's sign: no larger than what rounds to the largest number
  asm("min.xorsign.abs.f32 %0, %1, %2;" : "=f"(y) : "f"(x), "f"(__uint_as_float(0x7f7fefffu)));
  hi = (__float_as_uint(y) + 0x1000u) & 0xffffe000u;
  lo = __float_as_uint(x - __uint_as_float(hi));
}
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// four e4m3 codes as two pairs of f16: exact
__device__ __forceinline__ void e4m3x4_f16x4(uint32_t codes, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(codes));
}
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// ------------------------------------------------------------ configuration
// Keys of a warp's stage (one k step of bf16 and f32 products, two of e4m3's in
// f16: one takes 17% longer; at head_dim 256, where two make stages of 16 KB,
// one: two take 32% longer), its bytes (keys and values), warps and stages
// per CTA, CTAs per SM: about 200 KB of an SM's shared memory hold stages.
template <int KV, int DP>
struct AttnCfg {
  static constexpr int ES = kv_esize(KV);
  static constexpr int RB = DP * ES;             // bytes of a row
  static constexpr int KEYS = KV == MOE_KV_F32 ? 8 : KV == MOE_KV_BF16 || DP == 256 ? 16 : 32;
  static constexpr int NJ = KEYS / 8;
  static constexpr int SB = 2 * KEYS * RB;
  static constexpr int NW = SB == 16384 ? (KV == MOE_KV_F32 ? 5 : 6)
                            : KV == MOE_KV_F32 && DP == 128 ? 8 : 4;
  static constexpr int CTAS = SB == 16384 || NW == 8 ? 1 : SB == 8192 ? 2 : 3;
  static constexpr int ST = SB == 16384 ? 2 : SB == 8192 ? 3 : 4;
  static constexpr int THREADS = 32 * NW;
  // Weights are 2^(x - m): a logit x (base 2) more than LAG above the one that m
  // was taken from moves m, and that one itself has the weight 2^LIFT.  f16
  // weights (e4m3) need both: up to 2^15, they keep 11 bits down to 2^-27 of that
  // weight, and below it are off by 2^-38 of it at most, 2^-20 for 2^18 tokens;
  // without the lift they would end at 2^-25, which a token that takes nearly
  // all of the softmax leaves to a long context's others.
  static constexpr float LIFT = KV == MOE_KV_E4M3 ? 13.0f : 0.0f;
  static constexpr float LAG = KV == MOE_KV_E4M3 ? 2.0f : 8.0f;
  // what a unit's end and the next one's begin cost, in tiles (a batch of 64
  // with bf16, 180 MB: 56 us with 0, 45 with 1, 42 with 2 and 3; with f32, whose
  // tiles take longer, 92 us with 1, 95 with 2)
  static constexpr int END = KV == MOE_KV_F32 ? 1 : 2;
  static constexpr int TILE = NW * KEYS;
  // Q in shared memory unless its fragments fit registers; for f32 as two
  // terms, one after the other
  static constexpr bool QREG = KV != MOE_KV_F32 && DP <= 128;
  // row pitch of a term: conflict-free for ldmatrix (bf16) and for 8-byte
  // (f16) and 16-byte (f32) fragment loads
  static constexpr int QP = KV == MOE_KV_F32 ? DP * 4 + 64 : KV == MOE_KV_BF16 ? DP * 2 + 16 : DP * 2 + 32;
  static constexpr int QTERM = kRows * QP;
  static constexpr int QBYTES = QREG ? 0 : (KV == MOE_KV_F32 ? 2 : 1) * QTERM;
  static constexpr int RING = NW * ST * SB;
  static constexpr int SMEM = RING + QBYTES;
  // columns of O that fit a warp's stage as fp32 (joining the warps)
  static constexpr int JC = SB / (kRows * 4) < DP ? SB / (kRows * 4) : DP;
};

// 16-byte chunk `c` of row `r` within a 16-row block of RB-byte rows, swizzled
// so that the fragment loads of 8 rows hit all banks.  A warp's stage holds
// keys and values; f32 values use another pattern than f32 keys, because the
// value fragments take rows two apart.
template <int RB>
__device__ __forceinline__ uint32_t chunk_at(int r, int c, bool odd_first) {
  if constexpr (RB >= 128) {
    const int f = odd_first ? (((r & 1) << 2) | ((r >> 1) & 3)) : (r & 7);
    return r * RB + ((c ^ f) << 4);
  } else {
    return r * RB + ((c ^ ((r >> 1) & 3)) << 4);
  }
}

// ------------------------------------------------------------ the work list
__device__ __forceinline__ int2 span_of(const AttnArgs& A, int b, bool& cut) {
  int len = max(A.lens[b], 0);
  const long long room = static_cast<long long>(A.max_pages) * A.page;
  if (len > room) {
    len = static_cast<int>(room);
    cut = true;
  }
  return make_int2(A.window > 0 ? max(0, len - A.window) : 0, len);
}
__device__ __forceinline__ int tiles_of(int2 span, int tile) {
  return max(1, (span.y - span.x + tile - 1) / tile);
}

// A place in the CTA's range of tiles; every warp keeps one for the loads and
// one for the products.
struct Cursor {
  int b, x, t, nt;  // request, unit in request, tile in unit, tiles of a unit
  int first, len;   // the request's attended tokens
  long long left;   // places of the range from here on, units' ends included
};

// to the first tile of the next unit (left is the caller's business)
template <int TILE>
__device__ __forceinline__ void next_unit(Cursor& c, const AttnArgs& A, int units) {
  c.t = 0;
  if (++c.x < units) return;
  c.x = 0;
  ++c.b;
  if (c.left <= 0) return;
  bool cut = false;
  const int2 s = span_of(A, c.b, cut);
  c.first = s.x;
  c.len = s.y;
  c.nt = tiles_of(s, TILE);
}
template <int TILE, int END>
__device__ __forceinline__ void advance(Cursor& c, const AttnArgs& A, int units) {
  --c.left;
  if (++c.t < c.nt) return;
  c.left -= END;
  next_unit<TILE>(c, A, units);
}

// ln(sum 2^top), where weights are lifted by 2^lift: top without it and sum
// without it are both near what their rounding should be relative to
__device__ __forceinline__ float log_sum(float top, float sum, float lift) {
  if (sum == 0.0f) return -INFINITY;
  return ((top + lift) + log2f(sum * exp2f(-lift))) * 0.6931471805599453f;
}

template <int KV>
__device__ __forceinline__ void store4(void* out, long long at, float4 v) {
  if constexpr (KV == MOE_KV_F32) {
    *reinterpret_cast<float4*>(static_cast<float*>(out) + at) = v;
  } else {
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(out) + at) =
        make_uint2(bf16x2(v.x, v.y), bf16x2(v.z, v.w));
  }
}

template <int KV, int DP>
__global__ void __launch_bounds__(AttnCfg<KV, DP>::THREADS, AttnCfg<KV, DP>::CTAS)
    attn_decode_kernel(const AttnArgs A) {
  using C = AttnCfg<KV, DP>;
  constexpr int NW = C::NW, ST = C::ST, RB = C::RB, NT = DP / 8, NJ = C::NJ;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ long long s_sum[NW];
  __shared__ int s_b;
  __shared__ long long s_off;
  __shared__ int2 s_span;
  __shared__ uint32_t s_mask[NW][ST];
  __shared__ float s_m[NW][kRows], s_l[NW][kRows], s_q[kRows];
  constexpr uint32_t kAll = 0xffffffffu >> (32 - C::KEYS);  // a mask of live keys
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, c4 = lane & 3;
  const int units = A.heads * A.blocks;
  pdl_wait();
  pdl_trigger();

  // ---- this CTA's range of tiles
  bool cut = false;
  const int per = (A.B - 1) / C::THREADS + 1;
  const int b0 = static_cast<int>(min(static_cast<unsigned>(A.B), threadIdx.x * per));
  const int b1 = b0 + min(per, A.B - b0);  // (no sum passes an int)
  long long mine = 0;
  int2 last = make_int2(0, 0);
  for (int b = b0; b < b1; ++b) {
    last = span_of(A, b, cut);
    mine += tiles_of(last, C::TILE) + C::END;
  }
  long long incl = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += y;
  }
  if (lane == 31) s_sum[warp] = incl;
  __syncthreads();
  long long before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    if (w < warp) before += s_sum[w];
    total += s_sum[w];
  }
  total *= units;
  if (cut && A.err && blockIdx.x == 0) atomicOr(A.err, MOE_DEVERR_NO_SPACE);
  const int ctas = static_cast<int>(min(static_cast<long long>(gridDim.x), total));
  const int cta = blockIdx.x;
  if (threadIdx.x == 0) A.info[cta] = make_int4(0, 0, 0, 0);
  if (cta >= ctas) return;
  const long long begin = cta * total / ctas, end = (cta + 1) * total / ctas;
  {
    const long long lo = (before + incl - mine) * units, hi = (before + incl) * units;
    if (begin >= lo && begin < hi) {
      long long at = lo;
      int b = b0;
      int2 s = last;  // of the only request, where it is one
      for (; per > 1; ++b) {
        s = span_of(A, b, cut);
        const long long n = static_cast<long long>(tiles_of(s, C::TILE) + C::END) * units;
        if (begin < at + n) break;
        at += n;
      }
      s_b = b;
      s_span = s;
      s_off = begin - at;
    }
  }
  __syncthreads();
  Cursor cc;
  cc.b = s_b;
  {
    const int2 s = s_span;
    cc.first = s.x;
    cc.len = s.y;
    cc.nt = tiles_of(s, C::TILE);
    const int places = cc.nt + C::END;
    cc.x = static_cast<int>(s_off / places);
    cc.t = static_cast<int>(s_off - static_cast<long long>(cc.x) * places);
    cc.left = end - begin;
    if (cc.t >= cc.nt) {  // the range begins with a unit's end: on to the next
      cc.left -= places - cc.t;
      next_unit<C::TILE>(cc, A, units);
    }
  }
  Cursor lc = cc;
  bool bad_page = false;

  // ---- loads
  const uint32_t ring = static_cast<uint32_t>(__cvta_generic_to_shared(smem)) + warp * ST * C::SB;
  constexpr int CPR = RB / 16;                     // chunks of a row
  constexpr int RPI = CPR >= 32 ? 1 : 32 / CPR;    // rows per instruction
  constexpr int IPR = CPR > 32 ? CPR / 32 : 1;     // instructions per row
  const int chunks = A.dim * C::ES / 16;
  const long long lane_off =
      (RPI > 1 ? lane / CPR : 0) * A.s_token + (RPI > 1 ? lane % CPR : lane) * 16;
  struct Want {
    int row;   // row in the page of this lane's key (lanes 0 .. 15), -1: none
    int page;
  };
  // page id of this lane's key at cursor c
  auto want = [&](const Cursor& c) {
    Want w = {-1, 0};
    const int pos = c.first + c.t * C::TILE + warp * C::KEYS + lane % C::KEYS;
    if (c.left > 0 && pos < c.len) {
      const int p = A.page_shift >= 0 ? pos >> A.page_shift : pos / A.page;
      w.row = pos - p * A.page;
      w.page = __ldg(A.table + c.b * A.table_stride + p);
    }
    return w;
  };
  auto load = [&](const Cursor& c, const Want& w, int stage) {
    const bool in = w.page >= 0 && w.page < A.num_pages;
    bad_page |= w.row >= 0 && !in;
    const bool live = w.row >= 0 && in;
    const uint32_t mask = __ballot_sync(0xffffffffu, live) & kAll;
    if (lane == 0) s_mask[warp][stage] = mask;
    const uint32_t base = ring + stage * C::SB;
    if (mask) {
      const long long off =
          live ? w.page * A.s_page + w.row * A.s_token + (c.x / A.blocks) * A.s_head : 0;
      // rows that follow one another in one page: no row needs its own address
      const int row0 = __shfl_sync(0xffffffffu, w.row, 0);
      const int page0 = __shfl_sync(0xffffffffu, w.page, 0);
      const bool run = w.page == page0 && w.row == row0 + lane % C::KEYS;
      if (mask == kAll && __all_sync(0xffffffffu, run)) {
        const long long o = __shfl_sync(0xffffffffu, off, 0) + lane_off;
        const char *kp = A.k + o, *vp = A.v + o;
#pragma unroll
        for (int i = 0; i < C::KEYS / RPI; ++i) {
          const int r = i * RPI + (RPI > 1 ? lane / CPR : 0);
#pragma unroll
          for (int j = 0; j < IPR; ++j) {
            const int ch = (RPI > 1 ? lane % CPR : lane) + 32 * j;
            const bool real = ch < chunks;
            cp_async16(base + chunk_at<RB>(r, ch, true), real ? kp + 512 * j : A.k, real);
            cp_async16(base + C::KEYS * RB + chunk_at<RB>(r, ch, KV != MOE_KV_F32),
                       real ? vp + 512 * j : A.v, real);
          }
          kp += RPI * A.s_token;
          vp += RPI * A.s_token;
        }
      } else {
#pragma unroll 2
        for (int i = 0; i < C::KEYS / RPI; ++i) {
          const int r = i * RPI + (RPI > 1 ? lane / CPR : 0);
          const long long o = __shfl_sync(0xffffffffu, off, r);
          const bool row_live = (mask >> r) & 1u;
#pragma unroll
          for (int j = 0; j < IPR; ++j) {
            const int ch = (RPI > 1 ? lane % CPR : lane) + 32 * j;
            const bool real = row_live && ch < chunks;
            const long long at = o + (ch < chunks ? ch * 16 : 0);
            cp_async16(base + chunk_at<RB>(r, ch, true), A.k + at, real);
            cp_async16(base + C::KEYS * RB + chunk_at<RB>(r, ch, KV != MOE_KV_F32), A.v + at, real);
          }
        }
      }
    }
    cp_commit();
  };

  // the first ST - 1 stages: all their page ids are asked for before any use
  Want next = want(lc);
  {
    Want w[ST - 1];
    Cursor at = lc;
#pragma unroll
    for (int s = 0; s < ST - 1; ++s) {
      w[s] = next;
      if (lc.left > 0) advance<C::TILE, C::END>(lc, A, units);
      next = want(lc);
    }
#pragma unroll
    for (int s = 0; s < ST - 1; ++s) {
      load(at, w[s], s);
      if (at.left > 0) advance<C::TILE, C::END>(at, A, units);
    }
  }

  // ---- per-unit state
  float acc[NT][4];
  float m[2], l[2];
  uint32_t qf[C::QREG ? DP / 16 : 1][4];
  float sl = 0.0f, v_mul = 1.0f;  // logits' factor in base 2, values' factor
  float q_mul[2] = {1.0f, 1.0f};  // e4m3: power of two taken out of a row of Q
  int rows = 0, t_first = 0;
  int slot = 0;                   // stage of the products' tile
  const uint32_t qs = static_cast<uint32_t>(__cvta_generic_to_shared(smem)) + C::RING;

  while (cc.left > 0) {
    // ---- a unit (or the part of it in this range) begins: Q, m, l, O
    const int kvh = cc.x / A.blocks, h0 = kvh * A.group + (cc.x % A.blocks) * kRows;
    rows = min(kRows, (kvh + 1) * A.group - h0);
    t_first = cc.t;
    sl = A.scale_log2;
    if constexpr (KV == MOE_KV_E4M3) {
      sl *= A.k_scale[kvh];
      v_mul = A.v_scale[kvh];
    }
    if constexpr (KV == MOE_KV_F32) {
      const float* q = static_cast<const float*>(A.q) + cc.b * A.q_b + h0 * A.q_h;
      for (int i = threadIdx.x; i < kRows * (DP / 4); i += C::THREADS) {
        const int r = i / (DP / 4), d = i % (DP / 4) * 4;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < rows && d < A.dim) v = __ldg(reinterpret_cast<const float4*>(q + r * A.q_h + d));
        uint4 hi, lo;
        split_tf32(v.x, hi.x, lo.x);
        split_tf32(v.y, hi.y, lo.y);
        split_tf32(v.z, hi.z, lo.z);
        split_tf32(v.w, hi.w, lo.w);
        *reinterpret_cast<uint4*>(smem + C::RING + r * C::QP + d * 4) = hi;
        *reinterpret_cast<uint4*>(smem + C::RING + C::QTERM + r * C::QP + d * 4) = lo;
      }
      __syncthreads();
    } else {
      const __nv_bfloat16* q =
          static_cast<const __nv_bfloat16*>(A.q) + cc.b * A.q_b + h0 * A.q_h;
      // four neighbouring columns of a row as f16.  The row is first scaled by
      // a power of two that brings its largest value into [1, 2): bf16 has 8
      // bits and f16 11, nothing is rounded but what lies below 2^-17 of that
      auto as_f16 = [](uint2 v, float inv) {
        return make_uint2(f16x2(__uint_as_float(v.x << 16) * inv,
                                __uint_as_float(v.x & 0xffff0000u) * inv),
                          f16x2(__uint_as_float(v.y << 16) * inv,
                                __uint_as_float(v.y & 0xffff0000u) * inv));
      };
      auto largest = [](uint2 v) {
        return fmaxf(fmaxf(fabsf(__uint_as_float(v.x << 16)),
                           fabsf(__uint_as_float(v.x & 0xffff0000u))),
                     fmaxf(fabsf(__uint_as_float(v.y << 16)),
                           fabsf(__uint_as_float(v.y & 0xffff0000u))));
      };
      // (exponent of the scale, its inverse) for a row's largest value
      auto scale_of = [](float big, float& mul) {
        const int e = min(max(static_cast<int>(__float_as_uint(big) >> 23), 1), 253);
        mul = __uint_as_float(static_cast<uint32_t>(e) << 23);
        return __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
      };
      if constexpr (KV == MOE_KV_BF16 && C::QREG) {
        // fragments: rows g and g + 8, columns {2c, 2c+1} and {2c+8, 2c+9} of 16
#pragma unroll
        for (int kk = 0; kk < DP / 16; ++kk) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int r = g + (j & 1) * 8, d = 16 * kk + 2 * c4 + (j >> 1) * 8;
            qf[kk][j] = r < rows && d < A.dim
                               ? __ldg(reinterpret_cast<const unsigned int*>(q + r * A.q_h + d))
                               : 0u;
          }
        }
      } else if constexpr (KV == MOE_KV_BF16) {
        for (int r = warp; r < kRows; r += NW) {
#pragma unroll
          for (int j = 0; j < DP / 64; ++j) {
            const int d = 2 * (lane + 32 * j);
            *reinterpret_cast<uint32_t*>(smem + C::RING + r * C::QP + 2 * d) =
                r < rows && d < A.dim
                    ? __ldg(reinterpret_cast<const unsigned int*>(q + r * A.q_h + d))
                    : 0u;
          }
        }
        __syncthreads();
      } else if constexpr (C::QREG) {
        // keys come as 4 neighbouring codes per lane: lane c's columns of a
        // step of 16 are 4c .. 4c+3
        uint2 raw[DP / 16][2];
        float big[2] = {0.0f, 0.0f}, inv[2];
#pragma unroll
        for (int kk = 0; kk < DP / 16; ++kk) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int r = g + j * 8, d = 16 * kk + 4 * c4;
            raw[kk][j] = r < rows && d < A.dim
                             ? __ldg(reinterpret_cast<const uint2*>(q + r * A.q_h + d))
                             : make_uint2(0u, 0u);
            big[j] = fmaxf(big[j], largest(raw[kk][j]));
          }
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          big[j] = fmaxf(big[j], __shfl_xor_sync(0xffffffffu, big[j], 1));
          big[j] = fmaxf(big[j], __shfl_xor_sync(0xffffffffu, big[j], 2));
          inv[j] = scale_of(big[j], q_mul[j]);
        }
#pragma unroll
        for (int kk = 0; kk < DP / 16; ++kk)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint2 x = as_f16(raw[kk][j], inv[j]);
            qf[kk][j] = x.x;
            qf[kk][2 + j] = x.y;
          }
      } else {
        for (int r = warp; r < kRows; r += NW) {
          uint2 v[DP / 128];
          float big = 0.0f, mul;
#pragma unroll
          for (int j = 0; j < DP / 128; ++j) {
            const int d = 4 * (lane + 32 * j);
            v[j] = r < rows && d < A.dim ? __ldg(reinterpret_cast<const uint2*>(q + r * A.q_h + d))
                                         : make_uint2(0u, 0u);
            big = fmaxf(big, largest(v[j]));
          }
#pragma unroll
          for (int off = 16; off > 0; off >>= 1)
            big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, off));
          const float inv = scale_of(big, mul);
          if (lane == 0) s_q[r] = mul;
#pragma unroll
          for (int j = 0; j < DP / 128; ++j)
            *reinterpret_cast<uint2*>(smem + C::RING + r * C::QP + 8 * (lane + 32 * j)) =
                as_f16(v[j], inv);
        }
        __syncthreads();
        q_mul[0] = s_q[g];
        q_mul[1] = s_q[g + 8];
      }
    }
    // a logit is f s in base 2; a negative scale turns the sign of s instead,
    // so that the largest s is the largest logit
    const bool flip = sl < 0.0f;
    const float f[2] = {fabsf(sl) * q_mul[0], fabsf(sl) * q_mul[1]};
    m[0] = m[1] = -INFINITY;
    l[0] = l[1] = 0.0f;
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = 0.0f;

    // ---- the unit's tiles in this range
    bool more = true;
    Cursor unit = cc;
    while (more) {
      cp_wait<ST - 2>();
      __syncwarp();
      {  // refill the stage that was used last
        const int to = slot == 0 ? ST - 1 : slot - 1;
        const Cursor at = lc;
        const Want w = next;
        if (lc.left > 0) advance<C::TILE, C::END>(lc, A, units);
        next = want(lc);
        load(at, w, to);
      }
      const unsigned mask = s_mask[warp][slot];
      if (mask) {
        const uint32_t kb = ring + slot * C::SB, vb = kb + C::KEYS * RB;
        float s[NJ][4];
        if constexpr (KV == MOE_KV_F32) {
          // 3 products of (hi, lo) pairs; few terms to a chain: the tensor
          // cores cut, not round, their sums
          float hh[2][4] = {}, hl[2][4] = {};
#pragma unroll
          for (int kk = 0; kk < DP / 16; ++kk) {
            // lane c's columns of the two k = 8 steps: 4c, 4c+1 and 4c+2, 4c+3
            const uint32_t at = qs + g * C::QP + (4 * kk + c4) * 16;
            const uint4 ha = lds4(at), hb = lds4(at + 8 * C::QP);
            const uint4 la = lds4(at + C::QTERM), lb = lds4(at + C::QTERM + 8 * C::QP);
            const uint4 kv = lds4(kb + chunk_at<RB>(g, 4 * kk + c4, true));
            const uint32_t ah[2][4] = {{ha.x, hb.x, ha.y, hb.y}, {ha.z, hb.z, ha.w, hb.w}};
            const uint32_t al[2][4] = {{la.x, lb.x, la.y, lb.y}, {la.z, lb.z, la.w, lb.w}};
            uint32_t kh[4], kl[4];
            split_tf32(__uint_as_float(kv.x), kh[0], kl[0]);
            split_tf32(__uint_as_float(kv.y), kh[1], kl[1]);
            split_tf32(__uint_as_float(kv.z), kh[2], kl[2]);
            split_tf32(__uint_as_float(kv.w), kh[3], kl[3]);
            mma_tf32(hh[0], ah[0], kh[0], kh[1]);
            mma_tf32(hh[1], ah[1], kh[2], kh[3]);
            mma_tf32(hl[0], al[0], kh[0], kh[1]);
            mma_tf32(hl[1], ah[0], kl[0], kl[1]);
            mma_tf32(hl[0], al[1], kh[2], kh[3]);
            mma_tf32(hl[1], ah[1], kl[2], kl[3]);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) s[0][e] = hh[0][e] + hh[1][e] + (hl[0][e] + hl[1][e]);
        } else if constexpr (KV == MOE_KV_BF16) {
          float part[2][NJ][4] = {};  // even and odd steps: shorter chains
#pragma unroll
          for (int kk = 0; kk < DP / 16; ++kk) {
            uint32_t qa[4], r[4];
            if constexpr (C::QREG) {
#pragma unroll
              for (int j = 0; j < 4; ++j) qa[j] = qf[kk][j];
            } else {
              ldsm4(qs + ((lane & 7) + ((lane >> 3) & 1) * 8) * C::QP + (2 * kk + (lane >> 4)) * 16,
                    qa);
            }
            ldsm4(kb + chunk_at<RB>((lane & 7) + (lane >> 4) * 8, 2 * kk + ((lane >> 3) & 1), true),
                  r);
            mma_bf16(part[kk & 1][0], qa, r[0], r[1]);
            mma_bf16(part[kk & 1][1], qa, r[2], r[3]);
          }
#pragma unroll
          for (int j = 0; j < NJ; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[j][e] = part[0][j][e] + part[1][j][e];
        } else {
          float part[2][NJ][4] = {};  // even and odd steps: shorter chains
#pragma unroll
          for (int kk = 0; kk < DP / 16; kk += 2) {
            uint32_t qa[2][4];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              if constexpr (C::QREG) {
#pragma unroll
                for (int j = 0; j < 4; ++j) qa[t][j] = qf[kk + t][j];
              } else {
                const uint32_t at = qs + g * C::QP + (4 * (kk + t) + c4) * 8;
                const uint2 a = lds2(at), b = lds2(at + 8 * C::QP);
                qa[t][0] = a.x;
                qa[t][1] = b.x;
                qa[t][2] = a.y;
                qa[t][3] = b.y;
              }
            }
#pragma unroll
            for (int h = 0; h < C::KEYS / 16; ++h) {
              // x4: chunks kk and kk + 1 (16 columns each) of 16 keys
              uint32_t r[4], lo, hi;
              ldsm4(kb + chunk_at<RB>(16 * h + (lane & 7) + ((lane >> 3) & 1) * 8, kk + (lane >> 4),
                                      true),
                    r);
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                e4m3x4_f16x4(r[j], lo, hi);
                mma_f16(part[j >> 1][2 * h + (j & 1)], qa[j >> 1], lo, hi);
              }
            }
          }
#pragma unroll
          for (int j = 0; j < NJ; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[j][e] = part[0][j][e] + part[1][j][e];
        }
        // the running softmax: rows g (e = 0, 1) and g + 8 (e = 2, 3), keys
        // 8 j + 2 c + (e & 1); masked keys (their rows hold zeros) are left out
        if (flip) {
#pragma unroll
          for (int j = 0; j < NJ; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[j][e] = -s[j][e];
        }
        if (mask != kAll) {
#pragma unroll
          for (int j = 0; j < NJ; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (!((mask >> (8 * j + 2 * c4 + (e & 1))) & 1u)) s[j][e] = -INFINITY;
        }
        float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) top[e >> 1] = fmaxf(top[e >> 1], s[j][e]);
        bool grow = false;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 1));
          top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 2));
          // (-inf: every key of the row is masked here, or its logit is -inf)
          top[r] = top[r] == -INFINITY ? -INFINITY : top[r] * f[r];
          grow = grow || top[r] > m[r] + (C::LIFT + C::LAG);
        }
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            if (top[r] > m[r] + (C::LIFT + C::LAG)) {
              const float to = top[r] - C::LIFT;
              const float keep = ex2(m[r] - to);
              m[r] = to;
              l[r] *= keep;
#pragma unroll
              for (int i = 0; i < NT; ++i) {
                acc[i][2 * r] *= keep;
                acc[i][2 * r + 1] *= keep;
              }
            }
          }
        }
        // from here on the row has tokens, if only of logits -inf: m says so
        m[0] = fmaxf(m[0], -FLT_MAX);
        m[1] = fmaxf(m[1], -FLT_MAX);
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[j][e] = ex2(fmaf(s[j][e], f[e >> 1], -m[e >> 1]));
        if (mask != kAll) {
#pragma unroll
          for (int j = 0; j < NJ; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (!((mask >> (8 * j + 2 * c4 + (e & 1))) & 1u)) s[j][e] = 0.0f;
        }
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          l[0] += s[j][0] + s[j][1];
          l[1] += s[j][2] + s[j][3];
        }
        // ---- O += P V
        if constexpr (KV == MOE_KV_BF16) {
          // P as a sum of two bf16: 16 bits of it, where one would leave 8.
          // The second product is free: the tile's bytes take longer
          uint32_t ph[4], pl[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float x = s[j >> 1][(j & 1) * 2], y = s[j >> 1][(j & 1) * 2 + 1];
            ph[j] = bf16x2(x, y);
            pl[j] = bf16x2(x - __uint_as_float(ph[j] << 16),
                           y - __uint_as_float(ph[j] & 0xffff0000u));
          }
#pragma unroll
          for (int dd = 0; dd < DP / 16; ++dd) {
            uint32_t r[4];
            ldsm4t(vb + chunk_at<RB>((lane & 7) + ((lane >> 3) & 1) * 8, 2 * dd + (lane >> 4), true),
                   r);
            mma_bf16(acc[2 * dd], ph, r[0], r[1]);
            mma_bf16(acc[2 * dd + 1], ph, r[2], r[3]);
            mma_bf16(acc[2 * dd], pl, r[0], r[1]);
            mma_bf16(acc[2 * dd + 1], pl, r[2], r[3]);
          }
        } else if constexpr (KV == MOE_KV_E4M3) {
          // P rounded to f16: 2^-11 of each weight, as against the 2^-4 of the
          // cached values themselves (as pairs of f16, like bf16's: 147 us for
          // 256 requests up to 8192 where these take 129)
          uint32_t pt[C::KEYS / 16][4];
#pragma unroll
          for (int h = 0; h < C::KEYS / 16; ++h)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float* const x = s[2 * h + (j >> 1)] + (j & 1) * 2;
              pt[h][j] = f16x2(x[0], x[1]);
            }
          // x4: 16 columns of keys 0..7, 8..15, 16..23 and 24..31 (of 16 keys: two
          // times 16 columns).  A register holds codes (d, d+1), d = 2g, of keys
          // 2c and 2c + 1 of its 8: bytes 0 and 2 are column d of both keys,
          // bytes 1 and 3 column d + 1
          constexpr int kHalves = C::KEYS / 16;
#pragma unroll
          for (int ch = 0; ch < DP / 16; ch += 3 - kHalves) {
            uint32_t r[4], e[4], o[4];
            ldsm4t(vb + (kHalves == 2 ? chunk_at<RB>(lane, ch, true)
                                      : chunk_at<RB>(lane & 15, ch + (lane >> 4), true)),
                   r);
#pragma unroll
            for (int j = 0; j < 4; ++j) e4m3x4_f16x4(__byte_perm(r[j], 0, 0x3120), e[j], o[j]);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int at = 2 * (kHalves == 2 ? ch : ch + h);
              mma_f16(acc[at], pt[kHalves == 2 ? h : 0], e[2 * h], e[2 * h + 1]);
              mma_f16(acc[at + 1], pt[kHalves == 2 ? h : 0], o[2 * h], o[2 * h + 1]);
            }
          }
        } else {
          // lane c's two keys are 2c and 2c + 1, the very ones whose weights it
          // holds
          uint32_t ph[4], pl[4];
          split_tf32(s[0][0], ph[0], pl[0]);
          split_tf32(s[0][2], ph[1], pl[1]);
          split_tf32(s[0][1], ph[2], pl[2]);
          split_tf32(s[0][3], ph[3], pl[3]);
#pragma unroll
          for (int dd = 0; dd < DP / 32; ++dd) {
            float o[4][4] = {};
            const uint4 a = lds4(vb + chunk_at<RB>(2 * c4, 8 * dd + g, false));
            const uint4 b = lds4(vb + chunk_at<RB>(2 * c4 + 1, 8 * dd + g, false));
            const uint32_t va[4] = {a.x, a.y, a.z, a.w}, vb4[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
            for (int t = 0; t < 4; ++t) {
              uint32_t ah, al, bh, bl;
              split_tf32(__uint_as_float(va[t]), ah, al);
              split_tf32(__uint_as_float(vb4[t]), bh, bl);
              mma_tf32(o[t], pl, ah, bh);
              mma_tf32(o[t], ph, al, bl);
              mma_tf32(o[t], ph, ah, bh);
            }
            // the long sum over tiles in rounded fp32 additions
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
              for (int e = 0; e < 4; ++e) acc[4 * dd + t][e] += o[t][e];
          }
        }
      }
      more = cc.left > 1 && cc.t + 1 < cc.nt;
      if (more) {
        slot = slot + 1 == ST ? 0 : slot + 1;
        ++cc.t;
        --cc.left;
      }
    }

    // ---- the unit's part ends: join the warps through the stage just used
    // (its refill comes after the barrier below)
    const int t_last = cc.t;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
      if (c4 == 0) {
        s_m[warp][g + 8 * r] = m[r];
        s_l[warp][g + 8 * r] = l[r];
      }
    }
    const bool whole = t_first == 0 && t_last + 1 == unit.nt;
    const long long part = 2ll * cta + (t_first == 0 ? 0 : 1);
    constexpr int PASSES = DP / C::JC;
    float* const dump = reinterpret_cast<float*>(smem + (warp * ST + slot) * C::SB);
    __syncwarp();  // every lane is done with the stage
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
      if (p > 0) __syncthreads();
#pragma unroll
      for (int i = p * (NT / PASSES); i < (p + 1) * (NT / PASSES); ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int n = 2 * c4 + (e & 1);  // column of the instruction's result
          const int d = KV == MOE_KV_BF16   ? 8 * i + n
                        : KV == MOE_KV_E4M3 ? (i >> 1) * 16 + 2 * n + (i & 1)
                                            : (i >> 2) * 32 + 4 * n + (i & 3);
          dump[(g + 8 * (e >> 1)) * C::JC + d - p * C::JC] = acc[i][e];
        }
      __syncthreads();
      for (int i = threadIdx.x; i < rows * (C::JC / 4); i += C::THREADS) {
        const int r = i / (C::JC / 4), d = i % (C::JC / 4) * 4 + p * C::JC;
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < NW; ++w) top = fmaxf(top, s_m[w][r]);
        float sum = 0.0f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < NW; ++w) {
          const float k = top == -INFINITY ? 1.0f : ex2(s_m[w][r] - top);
          const float4 x = *reinterpret_cast<const float4*>(
              smem + (w * ST + slot) * C::SB + (r * C::JC + d - p * C::JC) * 4);
          sum += k * s_l[w][r];
          o.x += k * x.x;
          o.y += k * x.y;
          o.z += k * x.z;
          o.w += k * x.w;
        }
        if (whole) {
          // -inf: no tokens.  A sum of 0 over some (logits of -inf) leaves NaN
          const float inv = top == -INFINITY ? 0.0f : v_mul / sum;
          if (d < A.dim)
            store4<KV>(A.out, cc.b * A.o_b + (h0 + r) * A.o_h + d,
                       make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
          if (d == 0 && A.lse)
            A.lse[static_cast<long long>(cc.b) * A.Hq + h0 + r] = log_sum(top, sum, C::LIFT);
        } else {
          *reinterpret_cast<float4*>(A.part_o + (part * kRows + r) * DP + d) = o;
          if (d == 0) A.part_ml[part * kRows + r] = make_float2(top, sum);
        }
      }
    }
    if (threadIdx.x == 0 && t_last + 1 < unit.nt) {
      // the unit goes on in the next CTAs, up to the one whose range holds its
      // last tile: how many have a part of it, and this one's place among them
      const long long from = end - unit.left - t_first, to = from + unit.nt - 1;
      const int c0 = static_cast<int>(((from + 1) * ctas - 1) / total);
      const int c1 = static_cast<int>(((to + 1) * ctas - 1) / total);
      A.info[cta] = make_int4(cc.b, cc.x, c1 - c0 + 1, cta - c0);
    }
    __syncthreads();  // the stages and s_m may be used again
    slot = slot + 1 == ST ? 0 : slot + 1;
    advance<C::TILE, C::END>(cc, A, units);
  }
  cp_wait<0>();
  if (bad_page && A.err) atomicOr(A.err, MOE_DEVERR_BAD_PAGE);
}

// Joins the parts of the units that range borders cut: a unit that begins in
// CTA c and does not end there has c's first slot, then the second slots of the
// next CTAs.  Block c joins the unit that begins in CTA c if it has few parts, a
// row a warp.  The rows of a unit of many parts go to the blocks of all CTAs that
// it does not end in, whose warps take every 8th part, so that the loads of a
// long request's hundred parts are all in flight.  One block per CTA of the first
// kernel: all fit on the GPU at once (a block for each row and CTA, most without
// work, started in waves: 42 us instead of 38 for 64 requests up to 4096).  A
// part is loaded along with its maximum, a warp's rescaled to its own reference
// (all maxima first: one load more in the chain, 0.7 us of a short call's 7.9).
constexpr int kJoinWarps = 8;
constexpr int kFewParts = 8;
template <int KV, int DP>
__global__ void __launch_bounds__(32 * kJoinWarps) attn_join_kernel(const AttnArgs A) {
  constexpr int VL = DP / 32;  // columns per lane
  __shared__ float s_o[kJoinWarps][DP];
  __shared__ float s_m[kJoinWarps], s_l[kJoinWarps];
  pdl_wait();
  const int4 unit = A.info[blockIdx.x];
  const int parts = unit.z, cta = blockIdx.x - unit.w;
  const bool few = parts <= kFewParts;
  if (parts == 0 || (few && unit.w > 0)) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int kvh = unit.y / A.blocks, h0 = kvh * A.group + (unit.y % A.blocks) * kRows;
  const int rows = min(kRows, (kvh + 1) * A.group - h0);
  const float mul = KV == MOE_KV_E4M3 ? A.v_scale[kvh] : 1.0f;
  for (int r = few ? warp : unit.w; r < rows; r += few ? kJoinWarps : parts - 1) {
    auto at = [&](int p) { return (2ll * (cta + p) + (p == 0 ? 0 : 1)) * kRows + r; };
    auto load = [&](int p, float (&v)[VL]) {
      const float* x = A.part_o + at(p) * DP + lane * VL;
#pragma unroll
      for (int j = 0; j < VL; j += 2)
        *reinterpret_cast<float2*>(v + j) = *reinterpret_cast<const float2*>(x + j);
    };
    float top = -INFINITY, sum = 0.0f;
    float o[VL] = {};
    if (few) {
      const float2 ml = lane < parts ? A.part_ml[at(lane)] : make_float2(-INFINITY, 0.0f);
      float f = 0.0f;
#pragma unroll
      for (int p0 = 0; p0 < kFewParts; p0 += 4) {
        if (p0 >= parts) break;
        float v[4][VL];
#pragma unroll
        for (int p = 0; p < 4; ++p)
          if (p0 + p < parts) load(p0 + p, v[p]);
        if (p0 == 0) {  // with the first parts on their way
          top = ml.x;
#pragma unroll
          for (int off = 16; off > 0; off >>= 1)
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
          f = top == -INFINITY ? 1.0f : ex2(ml.x - top);
        }
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          if (p0 + p >= parts) break;
          const float g = __shfl_sync(0xffffffffu, f, p0 + p);
          sum += g * __shfl_sync(0xffffffffu, ml.y, p0 + p);
#pragma unroll
          for (int j = 0; j < VL; ++j) o[j] += g * v[p][j];
        }
      }
      const float inv = top == -INFINITY ? 0.0f : mul / sum;
      const long long to = unit.x * A.o_b + (h0 + r) * A.o_h + lane * VL;
      if constexpr (VL >= 4) {
#pragma unroll
        for (int j = 0; j < VL; j += 4)
          if (lane * VL + j < A.dim)
            store4<KV>(A.out, to + j,
                       make_float4(o[j] * inv, o[j + 1] * inv, o[j + 2] * inv, o[j + 3] * inv));
      } else {  // two lanes' columns together
        const float a = __shfl_down_sync(0xffffffffu, o[0], 1);
        const float b = __shfl_down_sync(0xffffffffu, o[1], 1);
        if (lane % 2 == 0 && lane * VL < A.dim)
          store4<KV>(A.out, to, make_float4(o[0] * inv, o[1] * inv, a * inv, b * inv));
      }
    } else {
      // a warp's parts by its own reference, then the warps by theirs
      constexpr int kOnce = VL > 4 ? 2 : 4;
      for (int p0 = warp; p0 < parts; p0 += kOnce * kJoinWarps) {
        float2 ml[kOnce];
        float v[kOnce][VL], t = top;
#pragma unroll
        for (int i = 0; i < kOnce; ++i) {
          const int p = p0 + i * kJoinWarps;
          ml[i] = make_float2(-INFINITY, 0.0f);
          if (p < parts) {
            ml[i] = A.part_ml[at(p)];
            load(p, v[i]);
          }
        }
#pragma unroll
        for (int i = 0; i < kOnce; ++i) t = fmaxf(t, ml[i].x);
        const float g = t == -INFINITY ? 1.0f : ex2(top - t);
        top = t;
        sum *= g;
#pragma unroll
        for (int j = 0; j < VL; ++j) o[j] *= g;
#pragma unroll
        for (int i = 0; i < kOnce; ++i) {
          if (p0 + i * kJoinWarps >= parts) break;
          const float f = t == -INFINITY ? 1.0f : ex2(ml[i].x - t);
          sum += f * ml[i].y;
#pragma unroll
          for (int j = 0; j < VL; ++j) o[j] += f * v[i][j];
        }
      }
#pragma unroll
      for (int j = 0; j < VL; ++j) s_o[warp][lane * VL + j] = o[j];
      if (lane == 0) {
        s_m[warp] = top;
        s_l[warp] = sum;
      }
      __syncthreads();
      float f[kJoinWarps];
      top = -INFINITY;
      sum = 0.0f;
#pragma unroll
      for (int w = 0; w < kJoinWarps; ++w) top = fmaxf(top, s_m[w]);
#pragma unroll
      for (int w = 0; w < kJoinWarps; ++w) {
        f[w] = top == -INFINITY ? 1.0f : ex2(s_m[w] - top);
        sum += f[w] * s_l[w];
      }
      const int d = threadIdx.x * 4;
      if (d < A.dim) {
        float v[4] = {};
#pragma unroll
        for (int w = 0; w < kJoinWarps; ++w)
#pragma unroll
          for (int j = 0; j < 4; ++j) v[j] += f[w] * s_o[w][d + j];
        const float inv = top == -INFINITY ? 0.0f : mul / sum;
        store4<KV>(A.out, unit.x * A.o_b + (h0 + r) * A.o_h + d,
                   make_float4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv));
      }
    }
    if (A.lse && (few ? lane : static_cast<int>(threadIdx.x)) == 0)
      A.lse[static_cast<long long>(unit.x) * A.Hq + h0 + r] =
          log_sum(top, sum, AttnCfg<KV, DP>::LIFT);
    if (!few) __syncthreads();  // s_o is used again
  }
}

// ------------------------------------------------------------ host
static int attn_dp(int dim) { return dim <= 64 ? 64 : dim <= 128 ? 128 : 256; }

template <int KV, int DP>
static cudaError_t launch_attn(const AttnArgs& a, int ctas, cudaStream_t st) {
  using C = AttnCfg<KV, DP>;
  auto* kern = attn_decode_kernel<KV, DP>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), C::SMEM, done);
  if (e != cudaSuccess) return e;
  e = launch_chained(kern, dim3(ctas), dim3(C::THREADS), C::SMEM, st, a);
  if (e != cudaSuccess) return e;
  // units of one tile are never cut: nothing to join
  long long longest = static_cast<long long>(a.max_pages) * a.page;
  if (a.window > 0 && a.window < longest) longest = a.window;
  if (longest <= C::TILE) return cudaSuccess;
  return launch_chained(attn_join_kernel<KV, DP>, dim3(ctas), dim3(32 * kJoinWarps), 0, st, a);
}

template <int KV>
static int attn_ctas_per_sm(int dp) {
  return dp == 64 ? AttnCfg<KV, 64>::CTAS : dp == 128 ? AttnCfg<KV, 128>::CTAS
                                                      : AttnCfg<KV, 256>::CTAS;
}
static int ctas_per_sm(int kv, int dp) {
  return kv == MOE_KV_F32    ? attn_ctas_per_sm<MOE_KV_F32>(dp)
         : kv == MOE_KV_BF16 ? attn_ctas_per_sm<MOE_KV_BF16>(dp)
                             : attn_ctas_per_sm<MOE_KV_E4M3>(dp);
}

template <int KV>
static cudaError_t launch_kv(int dp, const AttnArgs& a, int ctas, cudaStream_t st) {
  return dp == 64    ? launch_attn<KV, 64>(a, ctas, st)
         : dp == 128 ? launch_attn<KV, 128>(a, ctas, st)
                     : launch_attn<KV, 256>(a, ctas, st);
}

static size_t up256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_attn_workspace(int kv_dtype, int head_dim) {
  if (kv_dtype < MOE_KV_F32 || kv_dtype > MOE_KV_E4M3 || head_dim < 1 || head_dim > 256 ||
      head_dim % kv_dim_step(kv_dtype))
    return 0;
  const int dp = attn_dp(head_dim);
  const size_t n = static_cast<size_t>(sm_count()) * ctas_per_sm(kv_dtype, dp);
  return up256(n * sizeof(int4)) + up256(2 * n * kRows * sizeof(float2)) +
         2 * n * kRows * dp * sizeof(float);
}

int moe_attn_decode(const moe_kv_cache_t* cache, const void* q, long long q_stride_b,
                    long long q_stride_h, int B, int Hq, const int32_t* block_table,
                    int max_pages, long long table_stride, const int32_t* seq_lens, float scale,
                    int window, void* out, long long o_stride_b, long long o_stride_h, float* lse,
                    void* ws, size_t ws_bytes, uint32_t* err, void* stream) {
  const int rc = kv_cache_ok(cache);
  if (rc != MOE_OK) return rc;
  if (B < 0 || Hq < 1 || Hq % cache->kv_heads || Hq > (1 << 20) || max_pages < 1 ||
      table_stride < max_pages || window < 0 ||
      static_cast<long long>(max_pages) * cache->page_size > kMaxLen || q_stride_b < 0 || q_stride_h < 0 ||
      o_stride_b < 0 || o_stride_h < 0 || !std::isfinite(scale))
    return MOE_ERR_INVALID_ARG;
  if (B == 0) return MOE_OK;
  if (!q || !block_table || !seq_lens || !out || !ws) return MOE_ERR_INVALID_ARG;
  if (!apart(B, o_stride_b, cache->head_dim) || !apart(Hq, o_stride_h, cache->head_dim))
    return MOE_ERR_INVALID_ARG;
  const int qs = cache->kv_dtype == MOE_KV_F32 ? 4 : 2;
  if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(out) |
       static_cast<uintptr_t>(q_stride_b * qs) | static_cast<uintptr_t>(q_stride_h * qs) |
       static_cast<uintptr_t>(o_stride_b * qs) | static_cast<uintptr_t>(o_stride_h * qs)) &
      15)
    return MOE_ERR_UNSUPPORTED;
  if (reinterpret_cast<uintptr_t>(ws) & 255) return MOE_ERR_INVALID_ARG;
  const size_t need = moe_attn_workspace(cache->kv_dtype, cache->head_dim);
  if (ws_bytes < need) return MOE_ERR_WORKSPACE;
  const int sms = sm_count();
  if (sms < 1) return MOE_ERR_CUDA;
  const int es = kv_esize(cache->kv_dtype), dp = attn_dp(cache->head_dim);
  AttnArgs a = {};
  a.k = static_cast<const char*>(cache->k);
  a.v = static_cast<const char*>(cache->v);
  a.s_page = cache->stride_page * es;
  a.s_token = cache->stride_token * es;
  a.s_head = cache->stride_head * es;
  a.k_scale = cache->k_scale;
  a.v_scale = cache->v_scale;
  a.q = q;
  a.q_b = q_stride_b;
  a.q_h = q_stride_h;
  a.out = out;
  a.o_b = o_stride_b;
  a.o_h = o_stride_h;
  a.lse = lse;
  a.table = block_table;
  a.table_stride = table_stride;
  a.lens = seq_lens;
  a.err = err;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.B = B;
  a.Hq = Hq;
  a.heads = cache->kv_heads;
  a.group = Hq / cache->kv_heads;
  a.blocks = (a.group + kRows - 1) / kRows;
  a.dim = cache->head_dim;
  a.page = cache->page_size;
  a.page_shift = -1;
  for (int i = 0; i < 31; ++i)
    if (a.page == 1 << i) a.page_shift = i;
  a.num_pages = cache->num_pages;
  a.max_pages = max_pages;
  a.window = window;
  const int full = sms * ctas_per_sm(cache->kv_dtype, dp);
  uint8_t* w = static_cast<uint8_t*>(ws);
  a.info = reinterpret_cast<int4*>(w);
  w += up256(full * sizeof(int4));
  a.part_ml = reinterpret_cast<float2*>(w);
  w += up256(2ull * full * kRows * sizeof(float2));
  a.part_o = reinterpret_cast<float*>(w);
  // no more CTAs than the most tiles that these sizes can hold (of 32 tokens
  // at least; the kernel goes by the lengths themselves)
  long long longest = static_cast<long long>(max_pages) * cache->page_size;
  if (window > 0 && window < longest) longest = window;
  const long long units = static_cast<long long>(B) * a.heads * a.blocks;
  const long long per = (longest + 31) / 32;
  const int ctas = units >= full || per >= full || units * per >= full
                       ? full
                       : static_cast<int>(units * per);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = cache->kv_dtype == MOE_KV_F32    ? launch_kv<MOE_KV_F32>(dp, a, ctas, st)
                        : cache->kv_dtype == MOE_KV_BF16 ? launch_kv<MOE_KV_BF16>(dp, a, ctas, st)
                                                         : launch_kv<MOE_KV_E4M3>(dp, a, ctas, st);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
