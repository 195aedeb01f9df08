// sample.cu -- the next token of each row from its logits and one uniform
// random number (moe_sample, include/moe_route.h): temperature, top-k, min-p
// and top-p, then the draw by the running sum over the vocabulary.
//
// A token is chosen by where a sum passes a border, so two ways to add give
// two answers unless the sums are exact: weights are whole numbers of 2^-43
// of the largest one, right to 2^-35 of themselves, and added as
// 64-bit integers (in units of 2^-44).  A vocabulary of 2^18 stays below 2^63,
// and no order of additions, of CTAs or of atomics changes a sum.
//
// One cluster of C CTAs works on a row, each on a slice that it sweeps two or
// three times, the first from HBM and the others out of L2 (rows in flight
// are few enough to stay there); four CTAs share an SM, so one's waiting is
// another's work:
//   A  the largest logit (and its lowest index where the row is greedy)
//   B  with top-k or top-p: token counts by bins of width t / 256 below the
//      largest logit.  For a small top-k only the largest logits of groups of
//      tokens are counted, without a sweep: k of those in the bins down to one
//      bound the k-th token.  For top-p the counts times the bins' weights say
//      where the border lies, nearly; a window of bins around it with at most
//      256 tokens is chosen.
//   C  one sweep puts the window's tokens on a list and, where they are needed,
//      adds up the weights of all tokens and of those above the window.  The
//      first CTA sorts the list, one token a thread, and so finds the last kept
//      token exactly; the draw is among the list when nothing lies above it,
//      else it goes by the warps' sums, and the warp whose tokens it falls on
//      walks through them once more.
//      A border that the bins' weights put into the wrong bin is looked for once
//      more, beyond the window that the exact sums rule out.
//   D  where the border's bin alone has more than 256 tokens: equal ones, as is
//      usual with bf16, need their number only.  Others, or where there is no
//      such bin (top-p among the many that a large top-k left): the border is
//      narrowed to one logit value by histograms over order keys (at most
//      three), and ties count in index order.
// Rows without top-k and top-p only need their sums.
//
// Bound by latency for few rows (a dozen steps, each a few dependent loads or a
// cluster barrier), and for many that are greedy or have a small top-k: a CTA's
// loads, waited for in batches, and its barriers follow one another, and the
// other three CTAs of its SM do not fill the gaps (stalled warps per instruction
// issued: 12 by loads and 8 at barriers, greedy; 6 and 8, top-k).  By
// instructions where the whole vocabulary has to be weighed: 55 a token in all;
// 97 with the counts and the list of top-p, and the counts' shared-memory
// additions.  At 64 registers, which four CTAs an SM leave, the compiler spills:
// 420 bytes stored and 324 loaded a thread (f32), 520 and 432 (bf16).
// Measured on a GB300: one row of 131072 f32 with every restriction 12 us; 64 of
// 50257 bf16 with mixed ones 28 us; 512 of 131072 f32 greedy 60 us (4.4 TB/s of
// logits, 66% of the copy bandwidth), top-k 107, no restriction 170, top-p 281.
// With the rows' slices kept in shared memory (two CTAs an SM) greedy rows took
// 1.3 times as long, the others 1.4 to 2.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
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

namespace cg = cooperative_groups;

constexpr int kSampThreads = 256;
constexpr int kSampCtas = 4;    // per SM
constexpr int kSampWarps = kSampThreads / 32;
constexpr int kBins = 8192;     // of counts
constexpr int kPer = kBins / kSampThreads;            // a thread's: a coarse bin
constexpr int kBand = 512;      // bins of each of the two best bands (2 t wide)
constexpr int kCoarse = 16;     // bins in one where groups are counted
constexpr int kNear = 3 * kPer; // bins around the border among which the window lies
constexpr int kKeyBins = 2048;  // of D's histograms
constexpr float kBinsPerT = 256.0f;
constexpr float kBinStep = 0.99610137f;  // exp(-1 / kBinsPerT)
constexpr int kList = kSampThreads;  // tokens that the list holds: one a thread
constexpr int kGroups = 4;           // groups of tokens per thread
constexpr int kSmallK = 96;          // the largest top-k that starts from them
constexpr int kMaxCluster = 16;
constexpr int kMaxVocab = 1 << 18;

// Where bin b's count lies: so that threads read their kPer neighbouring bins,
// and tokens of neighbouring bins add to them, without bank conflicts
static_assert(kPer == 32 && (kBins & (kBins - 1)) == 0, "the swizzle below");
__device__ __forceinline__ int count_at(int b) { return (b ^ ((b >> 5) & 31)) & (kBins - 1); }

struct SampArgs {
  const void* logits;
  long long row_stride;
  const float* u;
  const float* temperature;
  const int* top_k;
  const float* top_p;
  const float* min_p;
  int* ids;
  float* probs;
  int V, slice;  // slice: elements per CTA
};

// round(2^(44 + j / 32))
__device__ const unsigned long long kPow2[32] = {
    17592186044416ull, 17977404757381ull, 18371058661769ull, 18773332464219ull, 19184414915921ull,
    19604498901178ull, 20033781527906ull, 20472464220127ull, 20920752812471ull, 21378857646762ull,
    21846993670708ull, 22325380538761ull, 22814242715178ull, 23313809579344ull, 23824315533396ull,
    24346000112214ull, 24879108095804ull, 25423889624159ull, 25980600314626ull, 26549501381838ull,
    27130859760289ull, 27724948229574ull, 28332045542385ull, 28952436555301ull, 29586412362452ull,
    30234270432094ull, 30896314746195ull, 31572855943056ull, 32264211463077ull, 32970705697691ull,
    33692670141585ull, 34430443548229ull};

// Order-preserving key of a finite logit (0 stands for none): as in routing
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t b = __float_as_uint(v == 0.0f ? 0.0f : v);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t u) {
  return __uint_as_float((u & 0x80000000u) ? (u & 0x7fffffffu) : ~u);
}

// x >> n, 0 for an n of 64 or more (a negative n is one)
__device__ __forceinline__ unsigned long long shift_right(unsigned long long x, int n) {
  unsigned long long y;
  asm("shr.u64 %0, %1, %2;" : "=l"(y) : "l"(x), "r"(n));
  return y;
}

// Two floats in a register pair, and what one instruction does to both
typedef unsigned long long F2;
__device__ __forceinline__ F2 f2(float a, float b) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 halves(F2 x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// What turns a logit l into its weight 2^x, x = (l - top) log2(e) / t, as a
// whole number of 2^-44 (an even one: rounded at 2^-43).  Every lane of the
// warp calls it, lane j holding T[j] = 2^(44 + j / 32).
//   x = k / 32 + r:  2^x = 2^(k >> 5) T[k & 31] (1 + (2^r - 1)),  |r| <= 2^-6,
// the table by rounding the powers themselves and 2^r - 1 by the first four terms
// of its Taylor series, with l - top, log2(e) / t and r each as the sum of two floats, and 2^r - 1 in
// fixed point of 2^-37: right to 2^-35 (two roundings to 2^-37, T's first 31
// bits, three roundings of the second degree's term).
struct Weigher {
  float top, ch, cl;    // c = log2(e) / t as a pair
  uint32_t t_hi, t_lo;  // T[lane], 45 bits

  __device__ __forceinline__ void set(float top_, float ch_, float cl_, unsigned long long T) {
    top = top_;
    ch = ch_;
    cl = cl_;
    t_hi = static_cast<uint32_t>(T >> 32);
    t_lo = static_cast<uint32_t>(T);
  }
  // of two logits, by the same operations on pairs of floats (512 rows of
  // 131072 with top-p: 303 -> 287 us).  A logit is at most top
  __device__ __forceinline__ void both(float l0, float l1, unsigned long long& w0,
                                       unsigned long long& w1) const {
    F2 z;
    const int2 E = fraction(l0, l1, z);
    w0 = whole(halves(z).x, E.x);
    w1 = whole(halves(z).y, E.y);
  }
  __device__ __forceinline__ unsigned long long operator()(float l) const {
    F2 z;
    const int E = fraction(l, l, z).x;
    return whole(halves(z).x, E);
  }

 private:
  // 2^r - 1 in units of 2^-37; z: k as the low bits of a float
  __device__ __forceinline__ int2 fraction(float l0, float l1, F2& z) const {
    constexpr float kRound = 12582912.0f;  // 1.5 2^23: x + kRound - kRound rounds x
    const F2 round = f2(kRound, kRound), back = f2(-kRound, -kRound), l32 = f2(32.0f, 32.0f);
    F2 rh, small;  // r = rh + small, rh exact
    const F2 l = f2(l0, l1), c = f2(ch, ch), t = f2(top, top), minus = f2(-1.0f, -1.0f);
    const F2 dh = add2(l, f2(-top, -top));
    const F2 b = fma2(l, minus, dh);  // (a product with -1 is exact)
    const F2 dl = fma2(add2(t, b), minus, fma2(fma2(b, minus, dh), minus, l));
    const F2 ph = mul2(dh, c);
    z = fma2(ph, l32, round);
    rh = fma2(add2(z, back), f2(-0.03125f, -0.03125f), ph);
    small = add2(fma2(dh, c, mul2(dh, f2(-ch, -ch))), fma2(dh, f2(cl, cl), mul2(dl, c)));
    // ln 2 as a pair, degrees 2 to 4 in floats
    constexpr float kC1 = 95265423360.0f, kC1l = -261.773682f;
    constexpr float kC2 = 33016479744.0f, kC3 = 7628426752.0f, kC4 = 1321905536.0f;
    const F2 C1 = f2(kC1, kC1), a = mul2(rh, C1);
    const F2 rest = fma2(small, C1,
                         fma2(rh, f2(kC1l, kC1l), fma2(rh, C1, mul2(rh, f2(-kC1, -kC1)))));
    const F2 r = add2(rh, small);
    const F2 q = fma2(fma2(r, f2(kC4, kC4), f2(kC3, kC3)), r, f2(kC2, kC2));
    const float2 x = halves(a), y = halves(fma2(q, mul2(r, r), rest));
    return make_int2(__float2int_rn(x.x) + __float2int_rn(y.x),
                     __float2int_rn(x.y) + __float2int_rn(y.y));
  }
  // What lies below 2^-45, -inf and NaN get 0: z's bits then stand for a shift
  // by more than 45 (the bits of floats ascend with them, a negative z or NaN
  // gives a negative shift, which counts as 2^32 less that), and the shift
  // leaves nothing, whatever the fraction's bits
  __device__ __forceinline__ unsigned long long whole(float z, int E) const {
    const int bits = __float_as_int(z);  // 0x4b400000 + k
    const uint32_t hi = __shfl_sync(0xffffffffu, t_hi, bits);
    const uint32_t lo = __shfl_sync(0xffffffffu, t_lo, bits);
    const long long T = static_cast<long long>((static_cast<unsigned long long>(hi) << 32) | lo);
    const int t31 = static_cast<int>(__funnelshift_r(lo, hi, 14));
    const unsigned long long w =
        static_cast<unsigned long long>(T + ((static_cast<long long>(t31) * E) >> 23));
    return (shift_right(w, (0x4b400000 >> 5) - (bits >> 5)) + 1ull) & ~1ull;
  }
};

// The same, called and not copied into the code: for passes that few rows take
__device__ __noinline__ unsigned long long weigh_call(const Weigher& w, float l) { return w(l); }

__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// adds 1 to shared memory where a < end: a predicate, not a branch
__device__ __forceinline__ void red_one(uint32_t addr, int a, int end) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.lt.s32 q, %1, %2;\n\t"
      "@q red.shared.add.u32 [%0], 1;\n\t}" ::"r"(addr),
      "r"(a), "r"(end)
      : "memory");
}

// floor(f n) for 0 <= f <= 1, and whether that is less than f n
__device__ __forceinline__ unsigned long long share_of(float f, unsigned long long n, bool& more) {
  const uint32_t b = __float_as_uint(f), e = b >> 23;
  more = false;
  if (e == 0) return 0;  // 0 (or below 2^-126)
  const unsigned long long m = (b & 0x7fffffu) | 0x800000u;
  const unsigned long long lo = n * m, hi = __umul64hi(n, m);
  const int sh = 150 - static_cast<int>(e);  // 23 .. 149
  if (sh < 64) {
    more = (lo & ((1ull << sh) - 1)) != 0;
    return (hi << (64 - sh)) | (lo >> sh);
  }
  const int s2 = min(sh - 64, 63);
  more = lo != 0 || (hi & ((1ull << s2) - 1)) != 0 || (hi >> s2 == 0 && hi != 0);
  return hi >> s2;
}

// What is kept (of the tokens that min-p keeps): order keys above one, and
// those equal to it up to an index
struct Cut {
  uint32_t key;
  int idx;
  __device__ __forceinline__ bool keeps(uint32_t k, int i) const {
    return k > key || (k == key && i <= idx);
  }
};

// What the first CTA finds, written into every CTA of the cluster
struct Result {
  int state;                  // 0 drawn already, 1 walk through warp `who`, 2 go to D,
                              // 3 another window, the border at `need`
  int who;
  uint32_t cut_key;
  int idx_cut;
  float need;
  int below;                  // of 3: the border is below the window, not above it
  unsigned long long before, total, to;
};

struct SampShared {
  union {
    alignas(16) uint32_t cnt[kBins];
    struct {
      uint32_t lo[kKeyBins], hi[kKeyBins];  // 64-bit sums of weights
    };
    struct {  // once all CTAs have read the counts
      unsigned long long list_x[kList], list_w[kList];
    };
  };
  float band[2][kSampWarps];  // what the bands' tokens weigh more than their bins
  alignas(8) float2 coarse[kSampThreads];  // count (as bits) and weight
  int near_n[kNear];  // the row's counts and weights around the border
  float near_w[kNear];
  // tokens of the window: ~order key << 32 | warp of the row << 18 | index, in
  // the order that they are kept in
  unsigned long long list[kList];
  alignas(16) unsigned long long all[kList];  // the row's (first CTA)
  int list_n;
  int cta_n[kMaxCluster];  // CTAs' counts (first CTA)
  unsigned long long kept;
  float edge[2];
  // by warp of the row, written by all CTAs into every one (tie, top) or the
  // first
  float warp_top[kMaxCluster * kSampWarps];
  int warp_tie[kMaxCluster * kSampWarps];
  uint2 warp_key[kMaxCluster * kSampWarps];
  unsigned long long warp_mass[kMaxCluster * kSampWarps];
  unsigned long long warp_all[kMaxCluster * kSampWarps];
  unsigned long long part_mass[kSampWarps];
  int cut_idx;
  Result result;
  long long scan[2 * kSampWarps];
  int at_bin, at_count, win_lo, win_hi, above_n;
  int near_above;
  float near_w_above, win_w;
  unsigned long long at_mass;
  unsigned long long key_sum[kSampThreads];
};

__device__ __forceinline__ int cut_to_int(long long v) {
  return v > INT_MAX ? INT_MAX : static_cast<int>(v);
}

// exclusive scan of two values over the CTA; also returns the totals
__device__ __forceinline__ void scan_pair(long long a, long long b, long long* sums,
                                          long long& ex_a, long long& ex_b, long long& tot_a,
                                          long long& tot_b) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long x = a, y = b;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, x, off);
    const long long v = __shfl_up_sync(0xffffffffu, y, off);
    if (lane >= off) {
      x += u;
      y += v;
    }
  }
  if (lane == 31) {
    sums[warp] = x;
    sums[kSampWarps + warp] = y;
  }
  __syncthreads();
  ex_a = x - a;
  ex_b = y - b;
  tot_a = tot_b = 0;
#pragma unroll
  for (int w = 0; w < kSampWarps; ++w) {
    if (w < warp) {
      ex_a += sums[w];
      ex_b += sums[kSampWarps + w];
    }
    tot_a += sums[w];
    tot_b += sums[kSampWarps + w];
  }
  __syncthreads();
}

// the same for a count and a weight, the weight's sums as they round in this order
__device__ __forceinline__ void scan_pair(int a, float b, long long* sums, int& ex_a, float& ex_b,
                                          float& tot_b) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = a;
  float y = b;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, x, off);
    const float v = __shfl_up_sync(0xffffffffu, y, off);
    if (lane >= off) {
      x += u;
      y += v;
    }
  }
  float2* const at = reinterpret_cast<float2*>(sums);
  if (lane == 31) at[warp] = make_float2(__int_as_float(x), y);
  __syncthreads();
  ex_a = x - a;
  ex_b = y - b;
  tot_b = 0.0f;
#pragma unroll
  for (int w = 0; w < kSampWarps; ++w) {
    const float2 v = at[w];
    if (w < warp) {
      ex_a += __float_as_int(v.x);
      ex_b += v.y;
    }
    tot_b += v.y;
  }
  __syncthreads();
}

__device__ __forceinline__ unsigned long long warp_sum(unsigned long long v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// The first `size` threads of a CTA (a power of two, 32 or more), as a group
// that orders and adds up one value a thread
__device__ __forceinline__ void group_sync(int size) {
  if (size == 32) __syncwarp();
  else named_bar_sync(1, size);
}

// the sum of the values before this thread's, and of all
__device__ __forceinline__ unsigned long long group_scan(unsigned long long x, int size,
                                                         unsigned long long* buf,
                                                         unsigned long long& all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  unsigned long long incl = x;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const unsigned long long y = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += y;
  }
  all = __shfl_sync(0xffffffffu, incl, 31);
  if (size == 32) return incl - x;
  if (lane == 31) buf[warp] = incl;
  group_sync(size);
  unsigned long long before = 0;
  all = 0;
  for (int w = 0; w < size / 32; ++w) {
    if (w < warp) before += buf[w];
    all += buf[w];
  }
  group_sync(size);
  return before + incl - x;
}

// A CTA's slice of the row as 16-byte chunks; a warp works on a run of them
template <typename LT>
struct Slice {
  static constexpr int VE = 16 / sizeof(LT);  // logits of a chunk
  const LT* base;  // chunk 0: 16-byte aligned, may begin before the slice
  int skip, stop;  // elements of the slice: skip <= i < stop, counted from base
  int first;       // index in the row of base's element
  int begin, end;  // this warp's chunks
  bool has_inf;    // +inf counts as the largest number

  // What does not belong to the slice reads as -inf, and nothing outside it is
  // touched
  __device__ __forceinline__ uint4 load(int c) const {
    constexpr uint32_t kNone = sizeof(LT) == 4 ? 0xff800000u : 0xff80ff80u;
    uint4 raw = make_uint4(kNone, kNone, kNone, kNone);
    if (c < end) {
      const int i = c * VE;
      if (i >= skip && i + VE <= stop) {
        raw = __ldg(reinterpret_cast<const uint4*>(base + i));
      } else {
        uint32_t w[4] = {kNone, kNone, kNone, kNone};
#pragma unroll
        for (int j = 0; j < VE; ++j)
          if (i + j >= skip && i + j < stop) {
            if constexpr (sizeof(LT) == 4) {
              w[j] = __float_as_uint(base[i + j]);
            } else {
              const uint32_t x = __bfloat16_as_ushort(base[i + j]);
              w[j / 2] = j % 2 ? (w[j / 2] & 0xffffu) | (x << 16) : (w[j / 2] & 0xffff0000u) | x;
            }
          }
        raw = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
    return raw;
  }

  // f(values, index of the first, number of the batch) for every chunk of this
  // warp, U loads at a time; all lanes stay together
  template <int U, typename F>
  __device__ __forceinline__ void sweep(F f) const {
    const int lane = threadIdx.x & 31;
    for (int c0 = begin; c0 < end; c0 += 32 * U) {
      uint4 raw[U];
#pragma unroll
      for (int i = 0; i < U; ++i) raw[i] = load(c0 + 32 * i + lane);
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
        float v[VE];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if constexpr (sizeof(LT) == 4) {
            v[j] = __uint_as_float(w[j]);
          } else {
            v[2 * j] = __uint_as_float(w[j] << 16);
            v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
          }
        }
        if (has_inf) {
          const float big = __uint_as_float(sizeof(LT) == 4 ? 0x7f7fffffu : 0x7f7f0000u);
#pragma unroll
          for (int j = 0; j < VE; ++j)
            if (v[j] == INFINITY) v[j] = big;
        }
        f(v, first + (c0 + 32 * i + lane) * VE, i);
      }
    }
  }
};

template <typename LT>
__global__ void __launch_bounds__(kSampThreads, kSampCtas) sample_kernel(const SampArgs A) {
  constexpr int VE = Slice<LT>::VE;
  constexpr int ES = sizeof(LT);
  constexpr int kFew = ES == 4 ? 2 : 1;  // chunks at a time where their tokens are weighed
  __shared__ SampShared S;
  cg::cluster_group cluster = cg::this_cluster();
  const int C = static_cast<int>(cluster.num_blocks());
  const int rank = static_cast<int>(cluster.block_rank());
  const int row = blockIdx.x / C;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int my_warp = rank * kSampWarps + warp, warps = C * kSampWarps;  // of the row
  const bool lead = rank == 0;
  auto everyone = [&]() {  // all threads of the row
    if (C > 1) cluster.sync();
    else __syncthreads();
  };
  const unsigned long long table = kPow2[lane];
  if (C > 1) cluster.barrier_arrive();  // waited for before the first write into another CTA
  pdl_wait();

  // ---- the row's settings, and the slice
  const float t = A.temperature ? A.temperature[row] : 1.0f;
  const int k_in = A.top_k ? A.top_k[row] : 0;
  const float p_in = A.top_p ? A.top_p[row] : 1.0f;
  const float min_p = A.min_p ? A.min_p[row] : 0.0f;
  const float u = fminf(fmaxf(A.u[row], 0.0f), 1.0f);  // NaN: 0
  const int k = k_in > 0 && k_in < A.V ? k_in : 0;
  const bool p_on = p_in < 1.0f;
  const float share = fmaxf(p_in, 0.0f);
  const bool min_on = t > 0.0f && min_p > 0.0f;
  Slice<LT> sl;
  int chunks, per_warp;  // of the slice
  {
    const int e0 = min(A.V, rank * A.slice), n = min(A.slice, A.V - e0);
    const LT* src = static_cast<const LT*>(A.logits) + row * A.row_stride + e0;
    sl.skip = static_cast<int>((reinterpret_cast<uintptr_t>(src) & 15) / ES);
    sl.base = src - sl.skip;
    sl.stop = sl.skip + n;
    sl.first = e0 - sl.skip;
    chunks = n > 0 ? (sl.stop + VE - 1) / VE : 0;
    per_warp = (chunks + kSampWarps - 1) / kSampWarps;
    sl.begin = min(chunks, warp * per_warp);
    sl.end = min(chunks, sl.begin + per_warp);
    sl.has_inf = false;
  }
  if (k || p_on)
    for (int i = tid; i < kBins; i += kSampThreads) S.cnt[i] = 0;
  if (tid == 0) {
    S.list_n = 0;
    S.at_bin = INT_MAX;
  }

  // ---- A: the largest logit (NaN is passed over; it never counts as >= any),
  // also of each of the thread's groups of tokens
  float group[kGroups];
#pragma unroll
  for (int i = 0; i < kGroups; ++i) group[i] = -INFINITY;
  sl.template sweep<8>([&](const float (&v)[VE], int, int i) {
#pragma unroll
    for (int j = 0; j < VE; ++j) group[i % kGroups] = fmaxf(group[i % kGroups], v[j]);
  });
  float top = group[0];
#pragma unroll
  for (int i = 1; i < kGroups; ++i) top = fmaxf(top, group[i]);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
  if (C > 1) {
    cluster.barrier_wait();
    if (lane < C) cluster.map_shared_rank(S.warp_top, lane)[my_warp] = top;
  } else if (lane == 0) {
    S.warp_top[my_warp] = top;
  }
  everyone();
  for (int i = lane; i < warps; i += 32) top = fmaxf(top, S.warp_top[i]);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
  if (top == -INFINITY) {  // nothing to draw
    if (lead && tid == 0) {
      A.ids[row] = -1;
      if (A.probs) A.probs[row] = 0.0f;
    }
    return;
  }
  if (top == INFINITY) {
    sl.has_inf = true;
    top = __uint_as_float(ES == 4 ? 0x7f7fffffu : 0x7f7f0000u);
#pragma unroll
    for (int i = 0; i < kGroups; ++i) group[i] = fminf(group[i], top);
  }
  if (!(t > 0.0f)) {  // greedy: the lowest index of the largest logit
    int idx = INT_MAX;
    if (S.warp_top[my_warp] != top && !sl.has_inf) sl.end = sl.begin;  // not here
    sl.template sweep<4>([&](const float (&v)[VE], int at, int) {
#pragma unroll
      for (int j = VE - 1; j >= 0; --j)
        if (v[j] == top) idx = min(idx, at + j);
    });
    idx = __reduce_min_sync(0xffffffffu, idx);
    if (lane == 0) cluster.map_shared_rank(S.warp_tie, 0)[my_warp] = idx;
    everyone();
    if (lead && warp == 0) {
      idx = INT_MAX;
      for (int i = lane; i < warps; i += 32) idx = min(idx, S.warp_tie[i]);
      idx = __reduce_min_sync(0xffffffffu, idx);
      if (lane == 0) {
        A.ids[row] = idx;
        if (A.probs) A.probs[row] = 1.0f;
      }
    }
    return;
  }
  Weigher weigh;
  {
    // log2(e) / t to 2^-46: quotient, and the remainder's quotient
    constexpr float kE = 1.44269502f, kEl = 1.92596299e-8f;  // log2(e)
    const float c = kE / t;
    weigh.set(top, fminf(c, 1e30f), c < 1e30f ? (fmaf(-c, t, kE) + kEl) / t : 0.0f, table);
  }
  // The lowest float for which `in`, which holds for the largest logit and for
  // every float above one for which it holds.  Each round of a warp tests 32 of
  // them, by order key; the first range is around an estimate, if its ends are
  // on both sides
  auto lowest = [&](float estimate, float off, auto in) {
    uint32_t lo = order_key(-FLT_MAX), hi = order_key(top);  // `in` holds for hi
    const float a = estimate - off, b = estimate + off;
    const unsigned both = __ballot_sync(0xffffffffu, in(fminf(lane ? b : a, top)));
    if (a > -FLT_MAX && !(both & 1u)) lo = order_key(a);
    if (b < top && (both & 2u)) hi = order_key(b);
    while (lo < hi) {
      const uint32_t step = (hi - lo + 31) / 32;
      const uint32_t key = min(hi, lo + step * lane);
      const unsigned reach = __ballot_sync(0xffffffffu, in(key_value(key)));
      const int j = reach ? __ffs(reach) - 1 : 32;
      hi = min(hi, lo + step * j);
      if (j > 0) lo = lo + step * (j - 1) + 1;
    }
    return key_value(hi);
  };
  float l_min = -FLT_MAX;  // the smallest logit that min-p keeps
  if (min_on) {
    // by the weights themselves
    bool more;
    const unsigned long long unit = 1ull << 44;
    unsigned long long least = share_of(fminf(min_p, 1.0f), unit, more);
    least = min(max(least + (more ? 1 : 0), 1ull), unit);
    const float at = t * logf(fminf(min_p, 1.0f));
    l_min = lowest(top + at, 1e-5f * (1.0f + fabsf(at) + fabsf(top)),
                   [&](float l) { return weigh(l) >= least; });
  }
  // bins of width t / 256 below the largest logit, the last one open;
  // monotonous in l, which is all that they have to be
  const float bin_scale = fminf(kBinsPerT / t, 1e30f);
  auto bin_at = [&](float z) {
    return __float_as_int(fminf(z, static_cast<float>(kBins - 1)) + 12582912.0f) - 0x4b400000;
  };
  auto bin_of = [&](float l) { return bin_at((top - l) * bin_scale); };
  // the first running sum of weights above u times their total is above this
  auto target = [&](unsigned long long total) {
    bool more;
    return min(share_of(u, total, more), total - 1);
  };
  // weights before a token for it to be out
  auto border_of = [&](unsigned long long total) {
    bool more;
    const unsigned long long b = share_of(share, total, more);
    return b + (more ? 1 : 0);
  };

  // ---- B: bins win_lo .. win_hi go to the list, those before are kept
  bool generic = false, dense = false;  // dense: the window is one bin, too full for the list
  bool weigh_all = !k, weigh_above = true;
  int win_lo = INT_MAX, win_hi = INT_MAX, above_n = 0;
  // The window for a border that lies `need` (2^-24 of the largest weight, as
  // the counts have it) or k tokens down, among the bins around it.  Where a
  // sweep has shown the exact border to lie below bin `after`, or above bin
  // `until`, it is taken from there on: the bins' weights are not exact
  int few = 0;                    // coarse bins whose tokens are half a list at most
  int near_c0 = -1, near_at = 0;  // first coarse bin of those, the border's among them
  auto choose = [&](float need, int after, int until) {
    if (warp == 0) {
      // one warp, kOne neighbouring bins a lane: the border's bin, then the
      // window: as many bins before it as 64 tokens allow (for top-k, whose
      // bin is exact, 256), as many after it as 128 in all allow
      constexpr int kOne = kNear / 32;
      int n[kOne], n_sum = 0;
      float w[kOne], w_sum = 0.0f;
#pragma unroll
      for (int i = 0; i < kOne; ++i) {
        n[i] = S.near_n[lane * kOne + i];
        w[i] = S.near_w[lane * kOne + i];
        n_sum += n[i];
        w_sum += w[i];
      }
      int n_at = n_sum;
      float w_at = w_sum;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, n_at, off);
        const float z = __shfl_up_sync(0xffffffffu, w_at, off);
        if (lane >= off) {
          n_at += y;
          w_at += z;
        }
      }
      n_at += S.near_above - n_sum;  // tokens before this lane's bins
      w_at += S.near_w_above - w_sum;
      after -= near_c0 * kPer;
      until -= near_c0 * kPer;
      unsigned at_i = (near_at + 1) * kPer - 1;  // where rounding hides the border
      if (static_cast<int>(at_i) <= after) at_i = kNear - 1;
      int last = -1;  // bin that has tokens and lies above `until`
      int n_i = n_at;
      float w_i = w_at;
#pragma unroll
      for (int i = 0; i < kOne; ++i) {
        const int b = lane * kOne + i;
        const bool hit = n[i] > 0 && b > after && (k ? n_i + n[i] >= k : w_i + w[i] >= need);
        if (hit) at_i = min(at_i, static_cast<unsigned>(b));
        if (n[i] > 0 && b < until) last = b;
        n_i += n[i];
        w_i += w[i];
      }
      int border = static_cast<int>(__reduce_min_sync(0xffffffffu, at_i));
      last = __reduce_max_sync(0xffffffffu, last);
      if (border >= until && last >= 0) border = last;
      int through = 0;  // tokens down to the border's bin, itself included
      n_i = n_at;
#pragma unroll
      for (int i = 0; i < kOne; ++i) {
        n_i += n[i];
        if (lane * kOne + i == border) through = n_i;
      }
      through = __reduce_max_sync(0xffffffffu, through);
      unsigned lo = border;
      n_i = n_at;
#pragma unroll
      for (int i = 0; i < kOne; ++i) {
        if (lane * kOne + i <= border && through - n_i <= (k ? kList : kList / 4))
          lo = min(lo, static_cast<unsigned>(lane * kOne + i));
        n_i += n[i];
      }
      lo = __reduce_min_sync(0xffffffffu, lo);
      int above = INT_MAX;
      n_i = n_at;
#pragma unroll
      for (int i = 0; i < kOne; ++i) {
        if (lane * kOne + i == static_cast<int>(lo)) above = n_i;
        n_i += n[i];
      }
      above = __reduce_min_sync(0xffffffffu, above);
      w_i = w_at;
#pragma unroll
      for (int i = 0; i < kOne; ++i) {
        if (lane * kOne + i == static_cast<int>(lo)) S.win_w = w_i;
        w_i += w[i];
      }
      int hi = border;
      n_i = n_at;
#pragma unroll
      for (int i = 0; i < kOne; ++i) {
        n_i += n[i];
        if (!k && n_i - above <= kList / 2) hi = max(hi, lane * kOne + i);
      }
      hi = __reduce_max_sync(0xffffffffu, hi);
      __syncwarp();
      if (lane == 0) {
        // few enough: all tokens from the largest logit on
        if (through <= (k ? kList : kList / 2)) {
          above = 0;
          S.win_w = 0.0f;
        }
        S.at_count = through - above;
        S.above_n = above;
        S.win_lo = above == 0 ? 0 : min(kBins - 1, near_c0 * kPer + static_cast<int>(lo));
        S.win_hi = min(kBins - 1, near_c0 * kPer + hi);
      }
    }
    __syncthreads();
    win_lo = S.win_lo;
    win_hi = S.win_hi;
    above_n = S.above_n;
    // a window from the largest logit on goes as far as its tokens allow, past
    // a gap that is wider than the bins around the border
    if (!k && above_n == 0 && S.at_count <= kList) win_hi = max(win_hi, few * kPer - 1);
  };
  if (k || p_on) {
    // groups, where there are well over k of them
    const bool small = k && k <= kSmallK && k * 4 <= min(C * kSampThreads * kGroups, A.V / VE);
    if (small) {
#pragma unroll
      for (int i = 0; i < kGroups; ++i)
        if (group[i] >= l_min) atomicAdd(&S.cnt[bin_of(group[i]) / kCoarse], 1u);
    } else {
      unsigned tail = 0;  // the last bin holds the far tail: added once
      float more[2] = {0.0f, 0.0f};  // the likeliest tokens' weights are not just their bin's
      const uint32_t counts = smem_u32(S.cnt);
      constexpr int kLast = 0x4b400000 + kBins - 1;  // bins as bits of 1.5 2^23 + b
      sl.template sweep<4>([&](const float (&v)[VE], int, int) {
        float z[VE], best = INFINITY;
        int bits[VE];
#pragma unroll
        for (int j = 0; j < VE; ++j) {
          z[j] = (top - v[j]) * bin_scale;  // NaN and -inf: in the last bin, not counted
          bits[j] = __float_as_int(fminf(z[j], static_cast<float>(kBins - 1)) + 12582912.0f);
          if (!(v[j] >= l_min)) bits[j] = kLast + 1;
          tail += bits[j] == kLast;
          red_one(counts + 4 * count_at(bits[j]), bits[j], kLast);
          best = fminf(best, z[j]);
        }
        if (!k && __any_sync(0xffffffffu, best < 2.0f * kBand)) {
          constexpr float kLog = -1.44269504f / kBinsPerT;
#pragma unroll
          for (int j = 0; j < VE; ++j) {
            const int b = bits[j] - 0x4b400000;
            const float e = ex2_approx(z[j] * kLog) - ex2_approx(static_cast<float>(b) * kLog);
            more[0] += b < kBand ? e : 0.0f;
            more[1] += b >= kBand && b < 2 * kBand ? e : 0.0f;
          }
        }
      });
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) {
        more[0] += __shfl_xor_sync(0xffffffffu, more[0], off);
        more[1] += __shfl_xor_sync(0xffffffffu, more[1], off);
      }
      if (lane < 2) S.band[lane][warp] = more[lane];
      tail = __reduce_add_sync(0xffffffffu, tail);
      if (lane == 0 && tail) atomicAdd(&S.cnt[count_at(kBins - 1)], tail);
      // coarse bins: this thread's kPer together
      __syncthreads();
      uint32_t n = 0;
      float w = 0.0f, scale = k ? 0.0f : exp2f(-1.44269504f / kBinsPerT * (tid * kPer));
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const uint32_t c = S.cnt[count_at(tid * kPer + i)];
        n += c;
        w = fmaf(static_cast<float>(c), scale, w);
        scale *= kBinStep;
      }
      // a band's correction counts from its end on
      if (!k && (tid + 1 == kBand / kPer || tid + 1 == 2 * kBand / kPer))
        for (int i = 0; i < kSampWarps; ++i) w += S.band[tid * kPer / kBand][i];
      S.coarse[tid] = make_float2(__uint_as_float(n), w);
    }
    everyone();
    int en;
    float ew, tw;
    if (small) {  // every CTA adds the counts up for itself
      constexpr int kTwo = kBins / kCoarse / kSampThreads;
      static_assert(kTwo == 2, "two coarse bins a thread");
      int cn[2] = {0, 0};
      uint2 x[kMaxCluster];
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r)
        x[r] = r < C ? reinterpret_cast<const uint2*>(cluster.map_shared_rank(S.cnt, r))[tid]
                     : make_uint2(0, 0);
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r) {
        cn[0] += x[r].x;
        cn[1] += x[r].y;
      }
      scan_pair(cn[0] + cn[1], 0.0f, S.scan, en, ew, tw);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (en < k && en + cn[i] >= k) S.at_bin = (2 * tid + i) * kCoarse + kCoarse - 1;
        en += cn[i];
      }
      __syncthreads();
      win_lo = 0;
      win_hi = min(S.at_bin, kBins - 1);
      weigh_above = false;
    } else {
      // every CTA adds the coarse bins up for itself, in the same order
      float2 x[kMaxCluster];
      float sw = 0.0f;
      int sn = 0;
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r)
        x[r] = r < C ? *cluster.map_shared_rank(S.coarse + tid, r) : make_float2(0.0f, 0.0f);
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r) {
        sn += __float_as_int(x[r].x);
        sw += x[r].y;
      }
      // in units of 2^-24 of the largest one: only the window's choice goes by them
      constexpr float kUnit = 16777216.0f;
      sw *= kUnit;
      scan_pair(sn, sw, S.scan, en, ew, tw);
      const float need = tw * share;  // before the border
      const bool here = sn > 0 && (k ? en + sn >= k : ew + sw >= need);
      if (here) atomicMin(&S.at_bin, tid);
      few = __syncthreads_count(en + sn <= kList / 2);
      const bool found = S.at_bin < kSampThreads;  // else top-k keeps everything
      const int c0 = found ? max(0, S.at_bin - 1) : 0;
      if (tid == c0) {
        S.near_above = en;
        S.near_w_above = ew;
      }
      // the bins around it, from all CTAs
      for (int i = tid; i < kNear; i += kSampThreads) {
        const int b = c0 * kPer + i;
        int n = 0;
        float w = 0.0f;
        if (b < kBins) {
          uint32_t x[kMaxCluster];
#pragma unroll
          for (int r = 0; r < kMaxCluster; ++r)
            x[r] = r < C ? *cluster.map_shared_rank(S.cnt + count_at(b), r) : 0;
#pragma unroll
          for (int r = 0; r < kMaxCluster; ++r) n += x[r];
          if (!k)
            w = static_cast<float>(n) * kUnit * exp2f(-1.44269504f / kBinsPerT * b);
        }
        S.near_n[i] = n;
        S.near_w[i] = w;
      }
      __syncthreads();
      near_c0 = c0;
      near_at = S.at_bin - c0;
      if (found) choose(need, -1, 2 * kBins);
      if (found) {
        dense = S.at_count > kList;
        generic = dense && k && p_on;
      } else {
        win_lo = 0;
        win_hi = kBins - 1;
        generic = __syncthreads_or(en + sn > kList) != 0 || !k;
      }
      weigh_above = above_n > 0;
    }
  }

  const bool list_on = k || p_on;
  unsigned long long w_mine = 0;  // this warp's kept weight, where no list is needed
  if (!list_on) {
    sl.template sweep<kFew>([&](const float (&v)[VE], int, int) {
#pragma unroll
      for (int j = 0; j < VE; j += 2) {
        unsigned long long w[2];
        weigh.both(v[j], v[j + 1], w[0], w[1]);
        w_mine += (v[j] >= l_min ? w[0] : 0) + (v[j + 1] >= l_min ? w[1] : 0);
      }
    });
    w_mine = warp_sum(w_mine);
  }
  // the lowest logit in the bins 0 .. b that min-p keeps; above the largest for
  // b < 0
  auto edge = [&](int b) {
    if (b < 0) return static_cast<float>(INFINITY);
    if (b >= kBins - 1) return l_min;
    const float width = 1.0f / bin_scale;
    return fmaxf(l_min, lowest(top - (static_cast<float>(b) + 0.5f) * width,
                               1e-5f * (1.0f + fabsf(top) + static_cast<float>(b) * width),
                               [&](float l) { return bin_of(l) <= b; }));
  };
  Cut cut = {0, INT_MAX};
  long long ties = LLONG_MAX;      // kept of the tokens equal to the cut
  bool alike = false;              // a dense bin holds one value
  unsigned long long above = 0, everything = 0;
  // a dense bin's first and last order key, and the sums, from the warps'
  auto dense_sums = [&](uint32_t& bin_lo, uint32_t& bin_hi) {
    above = everything = 0;
    bin_lo = 0xffffffffu;
    bin_hi = 0;
    for (int i = lane; i < warps; i += 32) {
      above += S.warp_mass[i];
      everything += S.warp_all[i];
      bin_lo = min(bin_lo, S.warp_key[i].x);
      bin_hi = max(bin_hi, S.warp_key[i].y);
    }
    above = warp_sum(above);
    everything = warp_sum(everything);
    bin_lo = __reduce_min_sync(0xffffffffu, bin_lo);
    bin_hi = __reduce_max_sync(0xffffffffu, bin_hi);
  };
  // The last kept token of the row's list, and the draw or the warp that it falls
  // on: by the first CTA's first `size` threads, x a token of each
  int tries = 0;
  auto pick = [&](int n_list, int n, int size, unsigned long long x) {
    above = everything = 0;
    for (int i = lane; i < warps; i += 32) {
      above += S.warp_mass[i];
      everything += S.warp_all[i];
    }
    above = warp_sum(above);
    everything = warp_sum(everything);
    // in order: each token's place is the number of those before it
    {
      const unsigned long long w = weigh(x == ~0ull ? top : key_value(~static_cast<uint32_t>(x >> 32)));
      int place = 0;
#pragma unroll 4
      for (int i = 0; i < n; i += 2) {  // beyond n: ~0
        const ulonglong2 y = *reinterpret_cast<const ulonglong2*>(S.all + i);
        place += (y.x < x) + (y.y < x);
      }
      if (x != ~0ull) {
        S.list_x[place] = x;
        S.list_w[place] = w;
      }
    }
    group_sync(size);
    const bool have = tid < n;
    x = have ? S.list_x[tid] : 0;
    const unsigned long long w = have ? S.list_w[tid] : 0;
    const uint32_t pos = static_cast<uint32_t>(x);
    const int better = above_n + tid;
    bool keep = have && (!k || better < k);
    unsigned long long* const buf = reinterpret_cast<unsigned long long*>(S.scan);
    unsigned long long kept_w;
    const unsigned long long ex = group_scan(keep ? w : 0, size, buf, kept_w);
    bool missed = n_list > kList;  // a list that ran over means D
    unsigned long long border = ~0ull;
    if (p_on) {
      const unsigned long long left = above + kept_w;
      border = border_of(k ? left : everything);
      missed = missed || (above_n > 0 && above >= border) || left < border;
      keep = keep && (better == 0 || above + ex < border);
    }
    // the last one that is kept
    if (keep && !(tid + 1 < n && (!k || better + 1 < k) && above + ex + w < border)) {
      S.kept = ex + w;
      S.result.cut_key = ~static_cast<uint32_t>(x >> 32);
      S.result.idx_cut = static_cast<int>(pos & 0x3ffffu);
    }
    const bool drawn = above_n == 0;  // the draw is among the list
    if (missed) {
      if (tid == 0) S.result.state = 2;
      if (tid == 0 && !k && n_list <= kList && tries < 2 && near_c0 >= 0) {
        // the window lay beside the border: its place by the exact sum
        S.result.state = 3;
        S.result.below = border > above;
        const float miss = border >= above ? static_cast<float>(border - above)
                                           : -static_cast<float>(above - border);
        S.result.need = S.win_w + miss * 9.5367432e-7f;  // 2^-44 to 2^-24
      }
    } else if (drawn) {
      if (have) {
        S.all[tid] = pos;
        S.list_w[tid] = keep ? w : 0;
      }
    } else if (keep) {
      atomicAdd(&S.warp_mass[pos >> 18], w);
    }
    group_sync(size);
    const unsigned long long total = above + S.kept;
    const unsigned long long to = target(total);
    if (!missed && drawn) {  // in order of the index
      if (tid == 0) S.result.state = 0;
      unsigned long long sum = 0;
#pragma unroll 4
      for (int i = 0; i < n; ++i) sum += static_cast<uint32_t>(S.all[i]) < pos ? S.list_w[i] : 0;
      if (keep && sum <= to && to < sum + w) {
        A.ids[row] = static_cast<int>(pos & 0x3ffffu);
        if (A.probs) A.probs[row] = static_cast<float>(w) / static_cast<float>(total);
      }
    } else if (!missed && warp == 0) {
      // the warps' sums, with the list's kept tokens: which one the draw falls on
      constexpr int kOne = kMaxCluster * kSampWarps / 32;
      unsigned long long m[kOne], incl = 0;
#pragma unroll
      for (int i = 0; i < kOne; ++i) {
        m[i] = lane * kOne + i < warps ? S.warp_mass[lane * kOne + i] : 0;
        incl += m[i];
      }
      const unsigned long long mine = incl;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const unsigned long long y = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += y;
      }
      unsigned long long sum = incl - mine;
#pragma unroll
      for (int i = 0; i < kOne; ++i) {
        if (sum <= to && to < sum + m[i]) {
          S.result.who = lane * kOne + i;
          S.result.before = sum;
        }
        sum += m[i];
      }
      if (lane == 0) {
        S.result.state = 1;
        S.result.total = total;
        S.result.to = to;
      }
    }
    group_sync(size);
    if (tid > 0 && tid < C) cluster.map_shared_rank(&S, tid)->result = S.result;
  };
  float from = 0.0f, down_to = 0.0f;  // the window's ends
  for (; list_on && !generic; ++tries) {
    // ---- C
    above = everything = 0;
    auto enlist = [&](float v, int idx) {
      const int at = atomicAdd(&S.list_n, 1);
      if (at < kList)
        S.list[at] = (static_cast<unsigned long long>(~order_key(v)) << 32) |
                     (static_cast<uint32_t>(my_warp) << 18) | static_cast<uint32_t>(idx);
    };
    if (warp < 2) {
      const float e = edge(warp ? win_hi : win_lo - 1);
      if (lane == 0) S.edge[warp] = e;
    }
    __syncthreads();
    from = S.edge[0];
    down_to = S.edge[1];
    if (weigh_all) {
      sl.template sweep<kFew>([&](const float (&v)[VE], int at, int) {
        bool in = false;
#pragma unroll
        for (int j = 0; j < VE; j += 2) {  // without branches: the weights' steps interleave
          unsigned long long w[2];
          weigh.both(v[j], v[j + 1], w[0], w[1]);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            everything += v[j + i] >= l_min ? w[i] : 0;
            above += v[j + i] >= from ? w[i] : 0;
            in |= v[j + i] >= down_to && !(v[j + i] >= from);
          }
        }
        if (in) {
#pragma unroll
          for (int j = 0; j < VE; ++j)
            if (v[j] >= down_to && !(v[j] >= from)) enlist(v[j], at + j);
        }
      });
    } else {
      const int end = sl.end;
      if (!weigh_above && S.warp_top[my_warp] < down_to) sl.end = sl.begin;  // none of this warp's
      sl.template sweep<4>([&](const float (&v)[VE], int at, int) {
        float most = v[0];
#pragma unroll
        for (int j = 1; j < VE; ++j) most = fmaxf(most, v[j]);
        // a chunk without a logit that reaches the window needs no closer look
        if (!__any_sync(0xffffffffu, most >= down_to)) return;
#pragma unroll
        for (int j = 0; j < VE; ++j) {
          const bool up = v[j] >= from;
          if (v[j] >= down_to && !up) enlist(v[j], at + j);
          if (weigh_above && __any_sync(0xffffffffu, up)) {
            const unsigned long long w = weigh_call(weigh, v[j]);
            above += up ? w : 0;
          }
        }
      });
      sl.end = end;
    }
    if (weigh_all || weigh_above) {
      above = warp_sum(above);
      everything = warp_sum(everything);
    }
    if (dense) break;
    if (lane == 0) {
      cluster.map_shared_rank(S.warp_mass, 0)[my_warp] = above;
      cluster.map_shared_rank(S.warp_all, 0)[my_warp] = everything;
    }
    __syncthreads();
    if (tid == 0) cluster.map_shared_rank(S.cta_n, 0)[rank] = S.list_n;
    everyone();
    if (lead) {
      // thread i takes the CTAs' i-th token; which order they come in does not matter
      int n_list = 0, from_cta = -1, from_at = 0;
      for (int r = 0; r < C; ++r) {
        const int n = S.cta_n[r];
        if (tid >= n_list && tid < n_list + n) {
          from_cta = r;
          from_at = tid - n_list;
        }
        n_list += n;
      }
      const bool have = from_cta >= 0 && from_at < kList;
      unsigned long long x = ~0ull;
      if (have) x = cluster.map_shared_rank(S.list, from_cta)[from_at];
      S.all[tid] = x;
      if (tid == 0) S.kept = 0;
      __syncthreads();
      const int n = min(n_list, kList);
      int size = 32;  // of the group that works on the list
      while (size < n) size *= 2;
      if (tid < size) pick(n_list, n, size, x);
    }
    everyone();
    const int state = S.result.state;
    if (state == 0) return;
    if (state == 1) break;
    generic = state == 2;
    if (state == 3) {
      const float need = S.result.need;
      if (tid == 0) S.list_n = 0;
      choose(need, S.result.below ? win_hi : -1, S.result.below ? 2 * kBins : win_lo);
      dense = S.at_count > kList;
      weigh_above = above_n > 0;
      everyone();
    }
  }

  // ---- D
  if (dense && !generic) {
    // the border lies in one bin, all of whose tokens are often alike (bf16):
    // then their number and the sums say everything
    uint32_t bin_lo = 0xffffffffu, bin_hi = 0;
    int n = 0;
    sl.template sweep<4>([&](const float (&v)[VE], int, int) {
#pragma unroll
      for (int j = 0; j < VE; ++j)
        if (v[j] >= down_to && !(v[j] >= from)) {
          bin_lo = min(bin_lo, order_key(v[j]));
          bin_hi = max(bin_hi, order_key(v[j]));
          ++n;
        }
    });
    bin_lo = __reduce_min_sync(0xffffffffu, bin_lo);
    bin_hi = __reduce_max_sync(0xffffffffu, bin_hi);
    n = __reduce_add_sync(0xffffffffu, n);
    if (lane < C) {
      cluster.map_shared_rank(S.warp_all, lane)[my_warp] = everything;
      cluster.map_shared_rank(S.warp_mass, lane)[my_warp] = above;
      cluster.map_shared_rank(S.warp_key, lane)[my_warp] = make_uint2(bin_lo, bin_hi);
      cluster.map_shared_rank(S.warp_tie, lane)[my_warp] = n;
    }
    everyone();
    w_mine = above;
    dense_sums(bin_lo, bin_hi);
    const long long border = k ? k : max(1ll, static_cast<long long>(border_of(everything)));
    const long long passed = k ? above_n : static_cast<long long>(above);
    bool missed = passed >= border;
    if (!missed && bin_lo == bin_hi) {
      const long long w = k ? 1 : static_cast<long long>(weigh_call(weigh, key_value(bin_lo)));
      missed = w == 0 || border - passed > w * S.at_count;
      if (!missed) {
        alike = true;
        cut.key = bin_lo;
        ties = (border - passed + w - 1) / w;
      }
    }
    generic = missed;  // the border is beside the bin
  }
  if ((generic || dense) && !alike) {
    // `narrow`: the order key, lo .. hi, where the count or the weight
    // of the keys from it up reaches `need`, or 0; the same in all CTAs.
    // Histograms over keys hi - 2^sh i, on ever fewer keys.  passed: what the
    // keys above hi come to, then those above the result
    auto narrow = [&](bool mass, long long need, uint32_t lo, uint32_t hi, long long& passed) {
      for (;;) {
        const int sh = max(0, 32 - __clz(hi - lo) - 11);  // 2^11 bins
        everyone();  // nobody reads the last histogram any more
        for (int i = tid; i < kKeyBins; i += kSampThreads) S.lo[i] = S.hi[i] = 0;
        __syncthreads();
        sl.template sweep<4>([&](const float (&v)[VE], int, int) {
          bool some = false;  // most chunks have none
#pragma unroll
          for (int j = 0; j < VE; ++j)
            some |= v[j] >= l_min && order_key(v[j]) >= lo && order_key(v[j]) <= hi;
          if (!__any_sync(0xffffffffu, some)) return;
#pragma unroll
          for (int j = 0; j < VE; ++j) {
            const uint32_t key = order_key(v[j]);
            const bool ok = v[j] >= l_min && key >= lo && key <= hi;
            if (__any_sync(0xffffffffu, ok)) {
              const int b = static_cast<int>((hi - key) >> sh);
              unsigned long long w = 1;
              if (mass) w = weigh_call(weigh, ok ? v[j] : top);
              if (ok && w) {
                const uint32_t add = static_cast<uint32_t>(w);
                const uint32_t old = atomicAdd(&S.lo[b], add);
                const uint32_t up = static_cast<uint32_t>(w >> 32) + (old + add < old ? 1u : 0u);
                if (up) atomicAdd(&S.hi[b], up);
              }
            }
          }
        });
        __syncthreads();
        // as in B: coarse bins of all CTAs first, then the fine ones of one
        constexpr int kMine = kKeyBins / kSampThreads;
        unsigned long long sum = 0;
#pragma unroll
        for (int i = 0; i < kMine; ++i)
          sum += (static_cast<unsigned long long>(S.hi[tid * kMine + i]) << 32) +
                 S.lo[tid * kMine + i];
        S.key_sum[tid] = sum;
        if (tid == 0) S.at_bin = -1;
        everyone();
        {
          unsigned long long x[kMaxCluster];
#pragma unroll
          for (int r = 0; r < kMaxCluster; ++r)
            x[r] = r < C ? *cluster.map_shared_rank(S.key_sum + tid, r) : 0;
          sum = 0;
#pragma unroll
          for (int r = 0; r < kMaxCluster; ++r) sum += x[r];
        }
        long long ex, unused, tot, tot_b;
        scan_pair(static_cast<long long>(sum), 0, S.scan, ex, unused, tot, tot_b);
        if (passed + ex < need && passed + ex + static_cast<long long>(sum) >= need) {
          S.at_bin = tid;
          S.at_mass = static_cast<unsigned long long>(passed + ex);
        }
        __syncthreads();
        if (S.at_bin < 0) return 0u;
        if (warp == 0) {
          unsigned long long w = 0;  // lane i: fine bin i
          if (lane < kMine) {
            const int i = S.at_bin * kMine + lane;
            for (int r = 0; r < C; ++r)
              w += (static_cast<unsigned long long>(*cluster.map_shared_rank(S.hi + i, r)) << 32) +
                   *cluster.map_shared_rank(S.lo + i, r);
          }
          unsigned long long incl = w;
#pragma unroll
          for (int off = 1; off < 32; off <<= 1) {
            const unsigned long long y = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += y;
          }
          const long long at = static_cast<long long>(S.at_mass + incl - w);
          const unsigned hit = __ballot_sync(
              0xffffffffu, lane < kMine && at < need && at + static_cast<long long>(w) >= need);
          __syncwarp();
          if (hit && lane == __ffs(hit) - 1) {
            S.at_bin = S.at_bin * kMine + lane;
            S.at_mass = static_cast<unsigned long long>(at);
          }
        }
        __syncthreads();
        passed = static_cast<long long>(S.at_mass);
        hi -= static_cast<uint32_t>(S.at_bin) << sh;
        __syncthreads();
        if (sh == 0) return hi;
        // keys of bf16 lie 2^16 apart, so a bin has one: those of negative
        // logits end in ones, one below where a positive hi's bins begin
        if (ES == 2 && sh <= 16) return (hi & 0x8000ffffu) == 0 ? hi - 1 : hi;
        lo = max(lo, hi - ((1u << sh) - 1u));
      }
    };
    // a sum over all tokens of the row, the same in all CTAs
    auto row_sum = [&](unsigned long long x) {
      x = warp_sum(x);
      everyone();
      if (lane < C) cluster.map_shared_rank(S.warp_all, lane)[my_warp] = x;
      everyone();
      x = 0;
      for (int i = lane; i < warps; i += 32) x += S.warp_all[i];
      return warp_sum(x);
    };
    const uint32_t key_min = order_key(l_min), key_top = order_key(top);
    long long passed = 0;
    uint32_t key_end = 0xffffffffu;  // w_mine has the weights of the keys above it
    if (!generic) {
      uint32_t bin_lo;
      dense_sums(bin_lo, key_end);
      const long long border = k ? k : max(1ll, static_cast<long long>(border_of(everything)));
      passed = k ? above_n : static_cast<long long>(above);
      cut.key = narrow(!k, border, bin_lo, key_end, passed);
      const long long w =
          k ? 1 : static_cast<long long>(weigh_call(weigh, key_value(cut.key ? cut.key : bin_lo)));
      generic = cut.key == 0 || w == 0;  // the border is beside the bin
      if (!generic) ties = (border - passed + w - 1) / w;
    }
    if (generic) {
      cut.key = 0;
      ties = LLONG_MAX;
      key_end = 0xffffffffu;
      w_mine = 0;
      passed = 0;
      if (k) {
        unsigned long long live = 0;
        sl.template sweep<4>([&](const float (&v)[VE], int, int) {
#pragma unroll
          for (int j = 0; j < VE; ++j) live += v[j] >= l_min;
        });
        if (row_sum(live) > static_cast<unsigned long long>(k)) {
          cut.key = narrow(false, k, key_min, key_top, passed);
          ties = k - passed;
        }
      }
      if (p_on) {
        unsigned long long x = 0;
        sl.template sweep<1>([&](const float (&v)[VE], int, int) {
#pragma unroll
          for (int j = 0; j < VE; ++j) {
            const bool ok = v[j] >= l_min && order_key(v[j]) > cut.key;
            const unsigned long long w = weigh_call(weigh, v[j]);
            x += ok ? w : 0;
          }
        });
        const unsigned long long over_cut = row_sum(x);
        const unsigned long long w_cut = weigh_call(weigh, cut.key ? key_value(cut.key) : top);
        const unsigned long long at_cut =
            cut.key ? w_cut * static_cast<unsigned long long>(ties) : 0;
        const unsigned long long border = max(1ull, border_of(over_cut + at_cut));
        if (border <= over_cut) {
          passed = 0;
          cut.key = narrow(true, static_cast<long long>(border), max(key_min, cut.key + 1), key_top,
                           passed);
          const unsigned long long w = weigh_call(weigh, key_value(cut.key));
          ties = static_cast<long long>((border - passed + w - 1) / w);
        } else {  // among top-k's ties
          ties = min(ties, static_cast<long long>((border - over_cut + w_cut - 1) / w_cut));
        }
      }
    }
    int here = 0;              // this warp's tokens equal to the cut
    unsigned long long x = 0;  // and the weights between it and key_end
    sl.template sweep<4>([&](const float (&v)[VE], int, int) {
      bool some = false;
#pragma unroll
      for (int j = 0; j < VE; ++j)
        some |= v[j] >= l_min && order_key(v[j]) >= cut.key && order_key(v[j]) <= key_end;
      if (!__any_sync(0xffffffffu, some)) return;
#pragma unroll
      for (int j = 0; j < VE; ++j) {
        const uint32_t key = order_key(v[j]);
        const bool ok = v[j] >= l_min && key > cut.key && key <= key_end;
        here += v[j] >= l_min && key == cut.key;
        if (__any_sync(0xffffffffu, ok)) {
          const unsigned long long w = weigh_call(weigh, v[j]);
          x += ok ? w : 0;
        }
      }
    });
    w_mine += warp_sum(x);
    here = __reduce_add_sync(0xffffffffu, here);
    everyone();  // the sums before have been read
    if (lane < C) cluster.map_shared_rank(S.warp_tie, lane)[my_warp] = here;
  }
  const unsigned long long w_cut = cut.key ? weigh_call(weigh, key_value(cut.key)) : 0;
  unsigned long long before, total, to;
  int who = -1;
  if (generic || dense || !list_on) {
    // every warp finds the one that the draw falls on.  A warp's tokens equal to
    // the cut count as far as there are `ties` left for them
    if (!alike) {
      if (lane < C) cluster.map_shared_rank(S.warp_mass, lane)[my_warp] = w_mine;
      everyone();
    }
    unsigned long long tied = 0;
    total = 0;
    for (int i = lane; i < warps; i += 32) {
      total += S.warp_mass[i];
      if (cut.key) tied += static_cast<unsigned>(S.warp_tie[i]);
    }
    total = warp_sum(total);
    if (cut.key) total += min(warp_sum(tied), static_cast<unsigned long long>(ties)) * w_cut;
    to = target(total);
    unsigned long long sum = 0;
    long long ties_left = ties;
    before = 0;
    for (int i0 = 0; i0 < warps; i0 += 32) {
      unsigned long long m = i0 + lane < warps ? S.warp_mass[i0 + lane] : 0;
      int n = 0, kept = 0;
      if (cut.key) {
        n = i0 + lane < warps ? S.warp_tie[i0 + lane] : 0;
        int upto = n;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, upto, off);
          if (lane >= off) upto += y;
        }
        kept = static_cast<int>(max(0ll, min(static_cast<long long>(n), ties_left - (upto - n))));
        m += static_cast<unsigned long long>(kept) * w_cut;
        ties_left -= __shfl_sync(0xffffffffu, upto, 31);
      }
      unsigned long long incl = m;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const unsigned long long y = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += y;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, sum + incl - m <= to && to < sum + incl);
      if (hit) {
        const int at = __ffs(hit) - 1;
        who = i0 + at;
        before = __shfl_sync(0xffffffffu, sum + incl - m, at);
        if (cut.key) {
          kept = __shfl_sync(0xffffffffu, kept, at);
          n = __shfl_sync(0xffffffffu, n, at);
          cut.idx = kept == n ? INT_MAX : -1 - kept;
        }
      }
      sum += __shfl_sync(0xffffffffu, incl, 31);
    }
  } else {
    const Result R = S.result;
    who = R.who;
    cut.key = R.cut_key;
    cut.idx = R.idx_cut;
    before = R.before;
    total = R.total;
    to = R.to;
  }
  if (who / kSampWarps != rank) return;
  if (cut.idx < -1) {  // of that warp's tokens equal to the cut so many are kept: up to which index
    if (warp == who % kSampWarps) {
      int left = -1 - cut.idx;
      sl.template sweep<1>([&](const float (&v)[VE], int at, int) {
        int hit = 0;
#pragma unroll
        for (int j = 0; j < VE; ++j) hit += v[j] >= l_min && order_key(v[j]) == cut.key;
        int incl = hit;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, incl, off);
          if (lane >= off) incl += y;
        }
        int n = incl - hit;
#pragma unroll
        for (int j = 0; j < VE; ++j)
          if (v[j] >= l_min && order_key(v[j]) == cut.key && ++n == left) S.cut_idx = at + j;
        left -= __shfl_sync(0xffffffffu, incl, 31);
      });
    }
    __syncthreads();
    cut.idx = S.cut_idx;
  }
  // ---- that warp's tokens once more: every warp of its CTA adds up an eighth
  // of them, and the one whose eighth the draw falls in walks through it
  {
    const int from = min(chunks, who % kSampWarps * per_warp), end = min(chunks, from + per_warp);
    const int part = (end - from + 32 * kSampWarps - 1) / (32 * kSampWarps) * 32;
    sl.begin = min(end, from + warp * part);
    sl.end = min(end, sl.begin + part);
  }
  auto kept_weight = [&](float v, int idx) {
    const bool ok = v >= l_min && cut.keeps(order_key(v), idx);
    const unsigned long long w = weigh(v);
    return ok ? w : 0ull;
  };
  unsigned long long in_part = 0;
  sl.template sweep<1>([&](const float (&v)[VE], int at, int) {
#pragma unroll
    for (int j = 0; j < VE; ++j) in_part += kept_weight(v[j], at + j);
  });
  in_part = warp_sum(in_part);
  if (lane == 0) S.part_mass[warp] = in_part;
  __syncthreads();
  for (int w = 0; w < warp; ++w) before += S.part_mass[w];
  if (!(before <= to && to < before + in_part)) return;
  sl.template sweep<1>([&](const float (&v)[VE], int at, int) {
    if (before > to) return;  // drawn
    unsigned long long w[VE], here = 0;
#pragma unroll
    for (int j = 0; j < VE; ++j) {
      w[j] = kept_weight(v[j], at + j);
      here += w[j];
    }
    unsigned long long incl = here;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const unsigned long long y = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += y;
    }
    unsigned long long sum = before + incl - here;
#pragma unroll
    for (int j = 0; j < VE; ++j) {
      if (sum <= to && to < sum + w[j]) {
        A.ids[row] = at + j;
        if (A.probs) A.probs[row] = static_cast<float>(w[j]) / static_cast<float>(total);
      }
      sum += w[j];
    }
    before += __shfl_sync(0xffffffffu, incl, 31);
  });
}

// The largest cluster for a row on the current device: 16 CTAs where one fits
// (more than the portable 8: asked once per device and type), 0 on an error
static int max_cluster(int logits_dtype) {
  static std::atomic<int> known[2][64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  std::atomic<int>& mine = known[logits_dtype][dev];
  int n = mine.load(std::memory_order_relaxed);
  if (n) return n;
  const void* kern = logits_dtype == MOE_LOGITS_F32
                         ? reinterpret_cast<const void*>(sample_kernel<float>)
                         : reinterpret_cast<const void*>(sample_kernel<__nv_bfloat16>);
  n = 8;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) ==
      cudaSuccess) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kMaxCluster);
    cfg.blockDim = dim3(kSampThreads);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kMaxCluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int fit = 0;
    if (cudaOccupancyMaxActiveClusters(&fit, kern, &cfg) == cudaSuccess && fit > 0)
      n = kMaxCluster;
  }
  cudaGetLastError();  // a refusal above leaves 8
  mine.store(n, std::memory_order_relaxed);
  return n;
}

}  // namespace moe

using namespace moe;

extern "C" {

int moe_sample(const void* logits, int logits_dtype, int B, int V, long long row_stride,
               const float* u, const float* temperature, const int32_t* top_k,
               const float* top_p, const float* min_p, int32_t* ids, float* probs, void* stream) {
  if (B < 0 || B > 65535 || V < 1 || V > kMaxVocab || row_stride < 0) return MOE_ERR_INVALID_ARG;
  if (logits_dtype != MOE_LOGITS_F32 && logits_dtype != MOE_LOGITS_BF16) return MOE_ERR_INVALID_ARG;
  if (B == 0) return MOE_OK;
  if (!logits || !u || !ids) return MOE_ERR_INVALID_ARG;
  const int es = logits_dtype == MOE_LOGITS_F32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(logits) & (es - 1)) return MOE_ERR_INVALID_ARG;
  // CTAs per row: so many that the rows in flight, four CTAs on each SM, take
  // no more than about 96 MB of the L2, and more while the GPU is not full and a
  // CTA has 2048 tokens at least
  const long long slots = static_cast<long long>(sm_count()) * kSampCtas;
  const long long bytes = static_cast<long long>(V) * es;
  const int most = max_cluster(logits_dtype);
  if (most < 1 || slots < 1) return MOE_ERR_CUDA;
  int cluster = 1;
  while (cluster < 8 && (B < slots / cluster ? B : slots / cluster) * bytes > 96ll << 20)
    cluster *= 2;
  while (cluster < most && static_cast<long long>(B) * cluster * 2 <= slots &&
         V >= 4096ll * cluster)
    cluster *= 2;
  const SampArgs a = {logits, row_stride, u, temperature, top_k, top_p, min_p, ids, probs, V,
                      (((V + cluster - 1) / cluster) + 7) / 8 * 8};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const dim3 grid(static_cast<unsigned>(B) * cluster);
  const cudaError_t e =
      logits_dtype == MOE_LOGITS_F32
          ? launch_cluster(sample_kernel<float>, grid, dim3(kSampThreads), cluster, 0, st, a)
          : launch_cluster(sample_kernel<__nv_bfloat16>, grid, dim3(kSampThreads), cluster, 0, st, a);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
