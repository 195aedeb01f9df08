// sample.cu -- the next token of each row from its logits and one uniform
// random number (moe_sample, include/moe_route.h): temperature, top-k, min-p
// and top-p, then the draw by the running sum over the vocabulary.
//
// A token is chosen by where a sum passes a border, so two ways to add give
// two answers unless the sums are exact: weights are whole numbers of 2^-44
// of the largest one (1), computed to about 2^-38 of themselves, and added as
// 64-bit integers.  A vocabulary of 2^18 stays below 2^63, and no order of
// additions, of CTAs or of atomics changes a sum.
//
// One cluster of C CTAs works on a row; each CTA reads its slice of the row
// once, into shared memory, and all further passes read it there:
//   A  the largest logit (and its lowest index where the row is greedy)
//   B  with top-k or top-p: token counts by bins of width t / 128 below the
//      largest logit.  For a small top-k only every thread's largest logit is
//      counted: k of those in the bins down to one bound the k-th token.  For
//      top-p the counts times the bins' weights say where the border lies,
//      nearly; a window of bins around it with at most 512 tokens is chosen.
//   C  one pass puts the window's tokens on a list and, where they are needed,
//      adds up the weights of all tokens and of those above the window.  The
//      first CTA ranks the list's tokens against each other, one a thread, and
//      so finds the last kept token exactly; the draw is among the list when
//      nothing lies above it, else it goes by the warps' sums, and the warp
//      whose tokens it falls on walks through them once more.
//   D  where the window does not hold the border (a bin with more than 512
//      tokens, a border the counts misjudged, top-p among more than 512 that
//      top-k left): the border is narrowed to one logit value by histograms
//      over order keys (at most three), and ties are counted in index order.
// Rows without top-k and top-p only need C's sums.  Bound by the row's bytes
// where top-k is small; where the whole vocabulary has to be weighed, by the
// weights' instructions (about 50 a token, once).
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

constexpr int kSampThreads = 512;
constexpr int kSampWarps = kSampThreads / 32;
constexpr int kBins = 4096;     // of counts; half as many of weights
constexpr int kKeyBins = 2048;  // of D's histograms
constexpr float kBinsPerT = 128.0f;
constexpr int kList = kSampThreads;  // tokens that the list holds: one a thread
constexpr int kSmallK = kList / 2;   // top-k that starts from the threads' largest
constexpr int kMaxCluster = 8;
constexpr int kMaxVocab = 1 << 18;
// bytes of the largest slice (f32, 2^18 tokens over 8 CTAs) and its edges
constexpr int kMaxSlice = kMaxVocab / kMaxCluster * 4 + 32;

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

// What turns a logit l into its weight 2^x, x = (l - top) log2(e) / t, as a
// whole number of 2^-44 (an even one: rounded at 2^-43).  Every lane of the
// warp calls it, lane j holding T[j] = 2^(44 + j / 32).
//   x = k / 32 + r:  2^x = 2^(k >> 5) T[k & 31] (1 + (2^r - 1)),  |r| <= 2^-6,
// with r as the sum of an exact float and a small one, and 2^r - 1 in fixed
// point of 2^-37: the sum is right to about 2^-38.
struct Weigher {
  float top, ch, cl;    // c = log2(e) / t as a pair
  float tg, tl;         // top c as a multiple of 2^-10 and the rest
  uint32_t t_hi, t_lo;  // T[lane] >> 14, and its low 14 bits
  bool near;            // |top c| < 2^12: l c itself is a float pair near tg

  __device__ __forceinline__ void set(float top_, float ch_, float cl_, unsigned long long T) {
    top = top_;
    ch = ch_;
    cl = cl_;
    t_hi = static_cast<uint32_t>(T >> 14);
    t_lo = static_cast<uint32_t>(T & 16383);
    const float p = top * ch;
    near = fabsf(p) < 4096.0f;
    tg = rintf(p * 1024.0f) * 0.0009765625f;
    tl = (p - tg) + fmaf(top, cl, fmaf(top, ch, -p));
  }
  // l is a number (not NaN), at most top
  __device__ __forceinline__ unsigned long long operator()(float l) const {
    constexpr float kRound = 12582912.0f;  // 1.5 2^23: x + kRound - kRound rounds x
    float rh, small, z;  // r = rh + small, rh exact; z: k as the low bits of a float
    bool live;           // below x = -46 the weight rounds to 0
    if (near) {
      const float p = l * ch;
      const float e = fmaf(l, ch, -p);  // exact
      const float d = fmaxf(p - tg, -47.0f);
      live = d > -46.0f;
      z = fmaf(d, 32.0f, kRound);
      rh = p - fmaf(z - kRound, 0.03125f, tg);  // the fma is exact: a multiple of 2^-10
      small = fmaf(l, cl, e - tl);
    } else {
      // large logits or a small t: from the difference, with its rounding error
      const float dh = l - top;
      const float b = dh - l;
      const float dl = (l - (dh - b)) - (top + b);
      const float ph = dh * ch;
      live = ph > -46.0f;
      const float at = live ? ph : 0.0f;
      z = fmaf(at, 32.0f, kRound);
      rh = fmaf(z - kRound, -0.03125f, at);
      small = live ? fmaf(dh, ch, -ph) + fmaf(dh, cl, dl * ch) : 0.0f;
    }
    const int k = __float_as_int(z) - 0x4b400000;
    // 2^r - 1 in units of 2^-37: ln 2 as a pair, degrees 2 to 4 in floats
    constexpr float kC1 = 95265423360.0f, kC1l = -261.773682f;
    constexpr float kC2 = 33016479744.0f, kC3 = 7628426752.0f, kC4 = 1321905536.0f;
    const float a = rh * kC1;
    const float rest = fmaf(small, kC1, fmaf(rh, kC1l, fmaf(rh, kC1, -a)));
    const float r = rh + small;
    const float q = fmaf(fmaf(r, kC4, kC3), r, kC2);
    const int E = __float2int_rn(a) + __float2int_rn(fmaf(q, r * r, rest));
    const uint32_t hi = __shfl_sync(0xffffffffu, t_hi, k);
    const uint32_t lo = __shfl_sync(0xffffffffu, t_lo, k);
    const long long T = (static_cast<long long>(hi) << 14) | lo;
    const unsigned long long w = static_cast<unsigned long long>(
        T + ((static_cast<long long>(static_cast<int>(hi)) * E) >> 23));
    const unsigned long long v = ((w >> ((-(k >> 5)) & 63)) + 1ull) & ~1ull;
    return live ? v : 0ull;
  }
};

// The same, called and not copied into the code: for passes that few rows take
__device__ __noinline__ unsigned long long weigh_call(const Weigher& w, float l) { return w(l); }

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

// What the first CTA finds, written into every CTA of the cluster
struct Result {
  int state;                  // 0 drawn already, 1 walk through warp `who`, 2 go to D
  int who;
  uint32_t cut_key;           // kept: order key above it, or equal and idx <= idx_cut
  int idx_cut;
  unsigned long long before, total, to;
};

struct SampShared {
  union {
    alignas(16) uint32_t cnt[kBins];
    struct {
      uint32_t lo[kKeyBins], hi[kKeyBins];  // 64-bit sums of weights
    };
  };
  uint32_t list_key[kList];
  uint32_t list_pos[kList];  // warp of the row << 18 | index: ordered by index
  unsigned long long all[kList], list_w[kList];  // the row's list (first CTA)
  int list_n, list_at, all_n;
  int next_kept[kSampWarps];
  // by warp of the row, written by all CTAs into every one (tie, top) or the
  // first
  float warp_top[kMaxCluster * kSampWarps];
  int warp_tie[kMaxCluster * kSampWarps];
  unsigned long long warp_mass[kMaxCluster * kSampWarps];
  unsigned long long warp_all[kMaxCluster * kSampWarps];
  uint32_t cut_pos;  // written by one CTA into every one
  Result result;
  long long scan[2 * kSampWarps];
  float fscan[kSampWarps];
  int at_bin, at_count, at_in, win_lo, win_hi, above_n;
  unsigned long long at_mass;
  float ch, cl, l_min, u, p, t;
  double d_min;
  int k, min_on;
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

__device__ __forceinline__ unsigned long long warp_sum(unsigned long long v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// The first `size` threads of a CTA (a power of two, 32 or more), as a group
// that sorts and adds up one value a thread
__device__ __forceinline__ void group_sync(int size) {
  if (size == 32) __syncwarp();
  else named_bar_sync(1, size);
}

// ascending; buf: one value a thread
__device__ __forceinline__ unsigned long long group_sort(unsigned long long x, int size,
                                                         unsigned long long* buf) {
  const int tid = threadIdx.x;
  for (int k = 2; k <= size; k *= 2) {
    for (int j = k / 2; j > 0; j /= 2) {
      unsigned long long y;
      if (j >= 32) {
        buf[tid] = x;
        group_sync(size);
        y = buf[tid ^ j];
        group_sync(size);
      } else {
        y = __shfl_xor_sync(0xffffffffu, x, j);
      }
      x = ((tid & j) == 0) == ((tid & k) == 0) ? min(x, y) : max(x, y);
    }
  }
  return x;
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

template <typename LT>
struct Slice {
  static constexpr int VE = 16 / sizeof(LT);  // logits of a 16-byte chunk
  const uint4* chunk;  // in shared memory
  int chunks;
  int first;           // index of chunk 0's first element (may lie before the slice)
  int begin, end;      // this warp's chunks

  __device__ __forceinline__ void get(int c, float (&v)[VE]) const {
    if (c >= end) {
#pragma unroll
      for (int j = 0; j < VE; ++j) v[j] = -INFINITY;
      return;
    }
    const uint4 raw = chunk[c];
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (sizeof(LT) == 4) {
        v[j] = __uint_as_float(w[j]);
      } else {
        v[2 * j] = __uint_as_float(w[j] << 16);
        v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
      }
    }
  }
};

template <typename LT>
__global__ void __launch_bounds__(kSampThreads, 2) sample_kernel(const SampArgs A) {
  constexpr int VE = Slice<LT>::VE;
  constexpr int ES = sizeof(LT);
  extern __shared__ __align__(16) uint8_t slice_smem[];
  __shared__ SampShared S;
  cg::cluster_group cluster = cg::this_cluster();
  const int C = static_cast<int>(cluster.num_blocks());
  const int rank = static_cast<int>(cluster.block_rank());
  const int row = blockIdx.x / C;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int my_warp = rank * kSampWarps + warp, warps = C * kSampWarps;  // of the row
  const bool lead = rank == 0;
  const unsigned long long table = kPow2[lane];
  cluster.barrier_arrive();  // waited for before the first write into another CTA
  pdl_wait();

  // ---- the slice: 16-byte chunks of the row; the elements of the first and
  // the last chunk that lie outside the slice become -inf.  A warp brings the
  // chunks that it works on
  const int e0 = min(A.V, rank * A.slice), n = min(A.slice, A.V - e0);
  const LT* src = static_cast<const LT*>(A.logits) + row * A.row_stride + e0;
  const int mis = static_cast<int>((reinterpret_cast<uintptr_t>(src) & 15) / ES);
  Slice<LT> sl;
  sl.chunk = reinterpret_cast<const uint4*>(slice_smem);
  sl.chunks = n > 0 ? (mis + n + VE - 1) / VE : 0;
  sl.first = e0 - mis;
  const int per_warp = (sl.chunks + kSampWarps - 1) / kSampWarps;
  sl.begin = min(sl.chunks, warp * per_warp);
  sl.end = min(sl.chunks, sl.begin + per_warp);
  for (int c = sl.begin + lane; c < sl.end; c += 32) {
    LT* dst = reinterpret_cast<LT*>(slice_smem) + c * VE;
    const int at = c * VE - mis;  // in the slice
    if (at >= 0 && at + VE <= n) {
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src + at)
                   : "memory");
    } else {
      for (int j = 0; j < VE; ++j) {
        LT v;
        if (at + j >= 0 && at + j < n) {
          v = src[at + j];
        } else if constexpr (ES == 4) {
          v = -INFINITY;
        } else {
          v = __ushort_as_bfloat16(0xff80);
        }
        dst[j] = v;
      }
    }
  }
  asm volatile("cp.async.commit_group;" ::: "memory");
  if (tid == 0) {  // the row's settings, while its logits are on their way
    const float t = A.temperature ? A.temperature[row] : 1.0f;
    const int k = A.top_k ? A.top_k[row] : 0;
    const float p = A.top_p ? A.top_p[row] : 1.0f;
    const float m = A.min_p ? A.min_p[row] : 0.0f;
    S.t = t;
    S.k = k > 0 && k < A.V ? k : 0;
    S.p = p;
    S.u = A.u[row];
    S.list_n = S.all_n = 0;
    S.min_on = 0;
    if (t > 0.0f) {
      // log2(e) / t to 2^-46: quotient, and the remainder's quotient
      constexpr float kE = 1.44269502f, kEl = 1.92596299e-8f;  // log2(e)
      const float c = kE / t;
      S.ch = c < 1e30f ? c : 1e30f;
      S.cl = c < 1e30f ? (fmaf(-c, t, kE) + kEl) / t : 0.0f;
      S.min_on = m > 0.0f;
      if (m > 0.0f) S.d_min = static_cast<double>(t) * log(fmin(static_cast<double>(m), 1.0));
    }
  }
  for (int i = tid; i < kBins; i += kSampThreads) S.cnt[i] = 0;
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncwarp();

  // ---- A: the largest logit (NaN is passed over; it never counts as >= any)
  float mine = -INFINITY;
  for (int c = sl.begin + lane; c < sl.end; c += 32) {
    float v[VE];
    sl.get(c, v);
#pragma unroll
    for (int j = 0; j < VE; ++j) mine = fmaxf(mine, v[j]);
  }
  {
    float m = mine;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    cluster.barrier_wait();
    if (lane < C) cluster.map_shared_rank(S.warp_top, lane)[my_warp] = m;
  }
  cluster.sync();
  float top = -INFINITY;
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
  if (top == INFINITY) {  // +inf counts as the largest number
    const float big = ES == 4 ? FLT_MAX : __uint_as_float(0x7f7f0000u);
    for (int c = sl.begin + lane; c < sl.end; c += 32) {
      float v[VE];
      sl.get(c, v);
#pragma unroll
      for (int j = 0; j < VE; ++j)
        if (v[j] == INFINITY) {
          if constexpr (ES == 4) reinterpret_cast<float*>(slice_smem)[c * VE + j] = big;
          else reinterpret_cast<uint16_t*>(slice_smem)[c * VE + j] = 0x7f7f;
        }
    }
    __syncwarp();
    mine = fminf(mine, big);
    top = big;
  }
  if (!(S.t > 0.0f)) {  // greedy: the lowest index of the largest logit
    int idx = INT_MAX;
    for (int c = sl.begin + lane; c < sl.end; c += 32) {
      float v[VE];
      sl.get(c, v);
#pragma unroll
      for (int j = VE - 1; j >= 0; --j)
        if (v[j] == top) idx = min(idx, sl.first + c * VE + j);
    }
    idx = __reduce_min_sync(0xffffffffu, idx);
    if (lane == 0) cluster.map_shared_rank(S.warp_tie, 0)[my_warp] = idx;
    cluster.sync();
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
  weigh.set(top, S.ch, S.cl, table);
  float l_min = -FLT_MAX;  // the smallest logit that min-p keeps
  if (S.min_on) {
    if (tid == 0) {  // exact tests around its estimate
      const double d = S.d_min;
      float lm = fminf(top, fmaxf(-FLT_MAX, static_cast<float>(top + d)));
      for (int i = 0; i < 4 && lm > -FLT_MAX; ++i) {
        const float below = key_value(order_key(lm) - 1);
        if (!(static_cast<double>(below) - top >= d)) break;
        lm = below;
      }
      for (int i = 0; i < 4 && lm < top; ++i) {
        if (static_cast<double>(lm) - top >= d) break;
        lm = key_value(order_key(lm) + 1);
      }
      S.l_min = lm;
    }
    __syncthreads();
    l_min = S.l_min;
  }
  const int k = S.k;
  const bool p_on = S.p < 1.0f;
  const float share = fmaxf(S.p, 0.0f);
  const float u = fminf(fmaxf(S.u, 0.0f), 1.0f);  // NaN: 0
  // bins of width t / 128 below the largest logit, the last one open;
  // monotonous in l, which is all that they have to be
  const float bin_scale = fminf(kBinsPerT / S.t, 1e30f);
  auto bin_of = [&](float l) {
    const float z = fminf((top - l) * bin_scale, static_cast<float>(kBins - 1));
    return __float_as_int(z + 12582912.0f) - 0x4b400000;
  };
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
  bool generic = false, weigh_all = !k, weigh_above = true;
  int win_lo = INT_MAX, win_hi = INT_MAX, above_n = 0;
  if (k || p_on) {
    // k of the threads' largest, where there are well over k of them
    const bool small = k && k <= kSmallK && k * 4ll * VE <= A.V;
    if (small) {  // one count a thread, eight bins together
      if (mine >= l_min) atomicAdd(&S.cnt[bin_of(mine) >> 3], 1u);
    } else {
      unsigned tail = 0;  // the last bin holds the far tail: added once
      for (int c0 = sl.begin; c0 < sl.end; c0 += 32) {
        float v[VE];
        sl.get(c0 + lane, v);
#pragma unroll
        for (int j = 0; j < VE; ++j) {
          if (v[j] >= l_min) {
            const int b = bin_of(v[j]);
            if (b == kBins - 1) ++tail;
            else atomicAdd(&S.cnt[b], 1u);
          }
        }
      }
      tail = __reduce_add_sync(0xffffffffu, tail);
      if (lane == 0 && tail) atomicAdd(&S.cnt[kBins - 1], tail);
    }
    if (tid == 0) {
      S.at_bin = kBins - 1;
      S.at_count = INT_MAX;
      S.win_lo = kBins;
      S.win_hi = -1;
    }
    cluster.sync();
    constexpr int PER = kBins / kSampThreads;
    static_assert(PER == 8, "two 16-byte loads a thread");
    int cn[PER] = {};
    long long en, ew, tn, tw;
    if (small) {  // a thread holds 8 bins' count in one
      uint32_t x[kMaxCluster];
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r)
        x[r] = r < C ? *cluster.map_shared_rank(S.cnt + tid, r) : 0;
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r) cn[0] += x[r];
      scan_pair(cn[0], 0, S.scan, en, ew, tn, tw);
      if (en < k && en + cn[0] >= k) S.at_bin = tid * PER + PER - 1;
    } else {
      // CTA r adds up the r-th part of the bins and puts the sums in all CTAs,
      // in place: nobody else reads or writes that part
      const int part = kBins / C;
      for (int i = rank * part + tid; i < (rank + 1) * part; i += kSampThreads) {
        uint32_t x[kMaxCluster], sum = 0;
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r)
          x[r] = r < C ? *cluster.map_shared_rank(S.cnt + i, r) : 0;
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r) sum += x[r];
        for (int r = 0; r < C; ++r) *cluster.map_shared_rank(S.cnt + i, r) = sum;
      }
      cluster.sync();
      {
        const uint4* from = reinterpret_cast<const uint4*>(S.cnt) + tid * 2;
        const uint4 x = from[0], y = from[1];
        cn[0] = x.x; cn[1] = x.y; cn[2] = x.z; cn[3] = x.w;
        cn[4] = y.x; cn[5] = y.y; cn[6] = y.z; cn[7] = y.w;
      }
      long long sn = 0;
      float sw = 0.0f, step = 0.0f;
#pragma unroll
      for (int i = 0; i < PER; ++i) sn += cn[i];
      if (!k) {
        // weights as whole numbers of 2^-24: only the window's choice goes by them
        step = 16777216.0f * exp2f(-1.44269504f / kBinsPerT * (tid * PER));
#pragma unroll
        for (int i = PER - 1; i >= 0; --i)
          sw = fmaf(sw, 0.99221794f, static_cast<float>(cn[i]));  // exp(-1 / 128)
        sw *= step;
      }
      scan_pair(sn, static_cast<long long>(sw), S.scan, en, ew, tn, tw);
      const float need = static_cast<float>(tw) * share;
      long long n_at = en;
      float w_at = static_cast<float>(ew);
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const float wi = static_cast<float>(cn[i]) * step;
        const bool here = k ? n_at < k && n_at + cn[i] >= k
                            : w_at <= need && w_at + wi >= need && cn[i] > 0;
        if (here) atomicMin(&S.at_bin, tid * PER + i);
        n_at += cn[i];
        w_at += wi;
        step *= 0.99221794f;
      }
    }
    __syncthreads();
    const int at_bin = S.at_bin;
    if (small) {
      win_lo = 0;
      win_hi = at_bin;
      weigh_above = false;
    } else {
      // the window: from as many bins before the border's as 256 tokens (for
      // top-k, whose bin is exact, 512) allow, to as many as 512 allow
      if (at_bin / PER == tid) {
        long long incl = en;
#pragma unroll
        for (int i = 0; i < PER; ++i)
          if (i <= at_bin % PER) incl += cn[i];
        S.at_count = cut_to_int(incl);
      }
      __syncthreads();
      const long long through = S.at_count;
      const int most = k ? kList : kList / 2;
      long long n_at = en;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        if (tid * PER + i <= at_bin && through - n_at <= most) atomicMin(&S.win_lo, tid * PER + i);
        n_at += cn[i];
      }
      __syncthreads();
      win_lo = min(S.win_lo, at_bin);
      if (win_lo / PER == tid) {
        long long ex = en;
#pragma unroll
        for (int i = 0; i < PER; ++i)
          if (i < win_lo % PER) ex += cn[i];
        S.above_n = cut_to_int(ex);
      }
      __syncthreads();
      above_n = S.above_n;
      n_at = en;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        n_at += cn[i];
        if (tid * PER + i >= win_lo && n_at - above_n <= kList) atomicMax(&S.win_hi, tid * PER + i);
      }
      __syncthreads();
      win_hi = k ? at_bin : S.win_hi;
      generic = win_hi < at_bin || through - above_n > kList;
      weigh_above = above_n > 0;
    }
  }

  const bool list_on = k || p_on;
  unsigned long long w_mine = 0;  // this warp's kept weight, where no list is needed
  if (!list_on) {
    for (int c0 = sl.begin; c0 < sl.end; c0 += 32) {
      float v[VE];
      sl.get(c0 + lane, v);
#pragma unroll
      for (int j = 0; j < VE; ++j) {
        const bool ok = v[j] >= l_min;
        const unsigned long long w = weigh(ok ? v[j] : top);
        w_mine += ok ? w : 0;
      }
    }
    w_mine = warp_sum(w_mine);
  } else if (!generic) {
    // ---- C
    unsigned long long above = 0, everything = 0;
    auto enlist = [&](float v, int idx) {
      const int at = atomicAdd(&S.list_n, 1);
      if (at < kList) {
        S.list_key[at] = order_key(v);
        S.list_pos[at] = (static_cast<uint32_t>(my_warp) << 18) | static_cast<uint32_t>(idx);
      }
    };
    if (weigh_all) {
      for (int c0 = sl.begin; c0 < sl.end; c0 += 32) {
        float v[VE];
        sl.get(c0 + lane, v);
#pragma unroll
        for (int j = 0; j < VE; ++j) {
          const bool ok = v[j] >= l_min;
          const unsigned long long w = weigh(ok ? v[j] : top);
          const int b = ok ? bin_of(v[j]) : INT_MAX;
          everything += ok ? w : 0;
          above += b < win_lo ? w : 0;
          if (b >= win_lo && b <= win_hi) enlist(v[j], sl.first + (c0 + lane) * VE + j);
        }
      }
    } else {
      // nothing below this logit can lie in the window's bins: a chunk without
      // one that reaches it needs no closer look
      const float reach =
          fmaxf(l_min, top - (static_cast<float>(win_hi) + 2.0f) / bin_scale);
      for (int c0 = sl.begin; c0 < sl.end; c0 += 32) {
        float v[VE];
        sl.get(c0 + lane, v);
        float most = v[0];
#pragma unroll
        for (int j = 1; j < VE; ++j) most = fmaxf(most, v[j]);
        if (!__any_sync(0xffffffffu, most >= reach)) continue;
#pragma unroll
        for (int j = 0; j < VE; ++j) {
          const int b = v[j] >= l_min ? bin_of(v[j]) : INT_MAX;
          if (b >= win_lo && b <= win_hi) enlist(v[j], sl.first + (c0 + lane) * VE + j);
          if (weigh_above && __any_sync(0xffffffffu, b < win_lo)) {
            const unsigned long long w = weigh_call(weigh, b < win_lo ? v[j] : top);
            above += b < win_lo ? w : 0;
          }
        }
      }
    }
    if (weigh_all || weigh_above) {
      above = warp_sum(above);
      everything = warp_sum(everything);
    }
    if (lane == 0) {
      cluster.map_shared_rank(S.warp_mass, 0)[my_warp] = above;
      cluster.map_shared_rank(S.warp_all, 0)[my_warp] = everything;
    }
    // this CTA's list to the end of the first one's; its order does not matter
    __syncthreads();
    if (tid == 0) S.list_at = atomicAdd(cluster.map_shared_rank(&S.all_n, 0), S.list_n);
    __syncthreads();
    if (tid < S.list_n && S.list_at + tid < kList)
      cluster.map_shared_rank(S.all, 0)[S.list_at + tid] =
          (static_cast<unsigned long long>(~S.list_key[tid]) << 32) | S.list_pos[tid];
    cluster.sync();
    int size = 32;  // of the group that works on the list
    const int n_list = S.all_n;  // (of the first CTA)
    while (size < min(n_list, kList)) size *= 2;
    if (lead && tid < size) {
      above = everything = 0;
      for (int i = lane; i < warps; i += 32) {
        above += S.warp_mass[i];
        everything += S.warp_all[i];
      }
      above = warp_sum(above);
      everything = warp_sum(everything);
      // in order: key descending, index ascending
      const bool have = tid < n_list;
      unsigned long long x = group_sort(have ? S.all[tid] : ~0ull, size, S.list_w);
      const uint32_t key = ~static_cast<uint32_t>(x >> 32), pos = static_cast<uint32_t>(x);
      unsigned long long w = weigh(have ? key_value(key) : top);
      if (!have) w = 0;
      const int better = above_n + tid;
      bool keep = have && (!k || better < k);
      unsigned long long* const buf = reinterpret_cast<unsigned long long*>(S.scan);
      unsigned long long kept_w, ex = group_scan(keep ? w : 0, size, buf, kept_w);
      bool missed = n_list > kList;  // a list that ran over means D
      if (p_on) {
        const unsigned long long left = above + kept_w;
        const unsigned long long border = border_of(k ? left : everything);
        missed = missed || (above_n > 0 && above >= border) || left < border;
        keep = keep && (better == 0 || above + ex < border);
        ex = group_scan(keep ? w : 0, size, buf, kept_w);
      }
      const unsigned long long total = above + kept_w;
      const unsigned long long to = target(total);
      if (missed || above_n == 0) {
        if (tid == 0) S.result.state = missed ? 2 : 0;
        if (!missed) {  // the draw is among the list, in order of the index
          S.list_w[tid] = w;
          x = keep ? (static_cast<unsigned long long>(pos) << 32) | static_cast<uint32_t>(tid)
                   : ~0ull;
          x = group_sort(x, size, S.all);
          group_sync(size);
          w = x == ~0ull ? 0 : S.list_w[static_cast<uint32_t>(x)];
          ex = group_scan(w, size, buf, kept_w);
          if (ex <= to && to < ex + w) {
            A.ids[row] = static_cast<int>((x >> 32) & 0x3ffffu);
            if (A.probs) A.probs[row] = static_cast<float>(w) / static_cast<float>(total);
          }
        }
      } else {
        // the last kept token of the list, and the warps' sums with the
        // list's kept tokens: which warp the draw falls on
        if (tid == 0) {
          S.result.state = 1;
          S.result.total = total;
          S.result.to = to;
        }
        const bool next = __shfl_down_sync(0xffffffffu, keep, 1);
        if (lane == 0) S.next_kept[warp] = keep;
        group_sync(size);
        const bool after = lane < 31 ? next : tid + 1 < size && S.next_kept[warp + 1];
        if (keep && !after) {
          S.result.cut_key = key;
          S.result.idx_cut = static_cast<int>(pos & 0x3ffffu);
        }
        if (keep) atomicAdd(&S.warp_mass[pos >> 18], w);
        group_sync(size);
        if (warp == 0) {
          unsigned long long sum = 0;
          for (int i0 = 0; i0 < warps; i0 += 32) {
            const unsigned long long m = i0 + lane < warps ? S.warp_mass[i0 + lane] : 0;
            unsigned long long incl = m;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
              const unsigned long long y = __shfl_up_sync(0xffffffffu, incl, off);
              if (lane >= off) incl += y;
            }
            if (sum + incl - m <= to && to < sum + incl) {
              S.result.who = i0 + lane;
              S.result.before = sum + incl - m;
            }
            sum += __shfl_sync(0xffffffffu, incl, 31);
          }
        }
      }
      group_sync(size);
      if (tid > 0 && tid < C) cluster.map_shared_rank(&S, tid)->result = S.result;
    }
    cluster.sync();
    if (S.result.state == 0) return;
    generic = S.result.state == 2;
  }

  struct {
    uint32_t key;
    int idx;
  } cut = {0, INT_MAX};
  if (generic) {
    // ---- D.  Histograms of counts or weights over order keys hi - 2^sh i
    auto clear = [&]() {
      cluster.sync();  // nobody reads the last one any more
      for (int i = tid; i < kBins; i += kSampThreads) S.cnt[i] = 0;
      __syncthreads();
    };
    // the bin where the count or the weight passes `need`; in all CTAs
    auto narrow = [&](bool mass, long long need, uint32_t lo, long long& passed) {
      uint32_t hi = order_key(top);
      passed = 0;  // count or weight of the keys above hi
      for (;;) {
        const int sh = max(0, 32 - __clz(hi - lo) - 11);  // 2^11 bins
        clear();
        for (int c0 = sl.begin; c0 < sl.end; c0 += 32) {
          float v[VE];
          sl.get(c0 + lane, v);
#pragma unroll
          for (int j = 0; j < VE; ++j) {
            const uint32_t key = order_key(v[j]);
            const bool ok = v[j] >= l_min && key >= lo && key <= hi;
            if (!__any_sync(0xffffffffu, ok)) continue;
            const int b = static_cast<int>((hi - key) >> sh);
            if (!mass) {
              if (ok) atomicAdd(&S.lo[b], 1u);
            } else {
              const unsigned long long w = weigh_call(weigh, ok ? v[j] : top);
              if (ok && w) {
                const uint32_t add = static_cast<uint32_t>(w);
                const uint32_t old = atomicAdd(&S.lo[b], add);
                atomicAdd(&S.hi[b], static_cast<uint32_t>(w >> 32) + (old + add < old ? 1u : 0u));
              }
            }
          }
        }
        if (tid == 0) S.at_bin = kKeyBins - 1;
        cluster.sync();
        constexpr int PER = kKeyBins / kSampThreads;
        long long cw[PER] = {}, sum = 0;
        for (int r = 0; r < C; ++r) {
          const SampShared* o = cluster.map_shared_rank(&S, r);
          const uint4 l = *reinterpret_cast<const uint4*>(&o->lo[tid * PER]);
          const uint4 h = *reinterpret_cast<const uint4*>(&o->hi[tid * PER]);
          cw[0] += (static_cast<long long>(h.x) << 32) + l.x;
          cw[1] += (static_cast<long long>(h.y) << 32) + l.y;
          cw[2] += (static_cast<long long>(h.z) << 32) + l.z;
          cw[3] += (static_cast<long long>(h.w) << 32) + l.w;
        }
#pragma unroll
        for (int i = 0; i < PER; ++i) sum += cw[i];
        long long ex, unused, tot, tot_b;
        scan_pair(sum, 0, S.scan, ex, unused, tot, tot_b);
        long long at = passed + ex;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          if (at < need && at + cw[i] >= need) {
            S.at_bin = tid * PER + i;
            S.at_mass = static_cast<unsigned long long>(at);
          }
          at += cw[i];
        }
        __syncthreads();
        passed = static_cast<long long>(S.at_mass);
        hi -= static_cast<uint32_t>(S.at_bin) << sh;
        __syncthreads();
        if (sh == 0) return hi;
        lo = max(lo, hi - ((1u << sh) - 1u));
      }
    };
    // a sum over all tokens of the row, the same in all CTAs
    auto row_sum = [&](unsigned long long x) {
      x = warp_sum(x);
      cluster.sync();
      if (lane < C) cluster.map_shared_rank(S.warp_all, lane)[my_warp] = x;
      cluster.sync();
      x = 0;
      for (int i = lane; i < warps; i += 32) x += S.warp_all[i];
      return warp_sum(x);
    };
    auto mass_above = [&](uint32_t key) {
      unsigned long long x = 0;
      for (int c0 = sl.begin; c0 < sl.end; c0 += 32) {
        float v[VE];
        sl.get(c0 + lane, v);
#pragma unroll
        for (int j = 0; j < VE; ++j) {
          const bool ok = v[j] >= l_min && order_key(v[j]) > key;
          const unsigned long long w = weigh_call(weigh, ok ? v[j] : top);
          x += ok ? w : 0;
        }
      }
      return row_sum(x);
    };
    auto count_of = [&]() {
      unsigned long long x = 0;
      for (int c0 = sl.begin; c0 < sl.end; c0 += 32) {
        float v[VE];
        sl.get(c0 + lane, v);
#pragma unroll
        for (int j = 0; j < VE; ++j) x += v[j] >= l_min;
      }
      return row_sum(x);
    };
    const uint32_t key_min = order_key(l_min);
    uint32_t cut_key = 0;
    long long ties = LLONG_MAX, passed;  // kept of the tokens equal to the cut
    if (k && count_of() > static_cast<unsigned long long>(k)) {
      cut_key = narrow(false, k, key_min, passed);
      ties = k - passed;
    }
    if (p_on) {
      const unsigned long long over_cut = mass_above(cut_key);
      const unsigned long long w_cut = weigh_call(weigh, cut_key ? key_value(cut_key) : top);
      const unsigned long long at_cut = cut_key ? w_cut * static_cast<unsigned long long>(ties) : 0;
      const unsigned long long border = max(1ull, border_of(over_cut + at_cut));
      if (border <= over_cut) {
        cut_key = narrow(true, static_cast<long long>(border), max(key_min, cut_key + 1), passed);
        const unsigned long long w = weigh_call(weigh, key_value(cut_key));
        ties = static_cast<long long>((border - passed + w - 1) / w);
      } else {  // among top-k's ties
        ties = min(ties, static_cast<long long>((border - over_cut + w_cut - 1) / w_cut));
      }
    }
    // the index of the last kept tie
    int here = 0;
    for (int c0 = sl.begin; c0 < sl.end; c0 += 32) {
      float v[VE];
      sl.get(c0 + lane, v);
#pragma unroll
      for (int j = 0; j < VE; ++j) here += v[j] >= l_min && order_key(v[j]) == cut_key;
    }
    here = __reduce_add_sync(0xffffffffu, here);
    if (lane < C) cluster.map_shared_rank(S.warp_tie, lane)[my_warp] = here;
    if (tid == 0) S.cut_pos = INT_MAX;
    cluster.sync();
    long long before = 0;
    for (int i = lane; i < my_warp; i += 32) before += S.warp_tie[i];
    before = static_cast<long long>(warp_sum(static_cast<unsigned long long>(before)));
    if (before < ties && before + here >= ties) {
      int left = static_cast<int>(ties - before);  // the left-th tie of this warp
      for (int c0 = sl.begin; c0 < sl.end && left > 0; c0 += 32) {
        float v[VE];
        sl.get(c0 + lane, v);
        int hit = 0;
#pragma unroll
        for (int j = 0; j < VE; ++j) hit += v[j] >= l_min && order_key(v[j]) == cut_key;
        int incl = hit;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, incl, off);
          if (lane >= off) incl += y;
        }
        if (incl >= left && incl - hit < left) {
          int at = incl - hit;
#pragma unroll
          for (int j = 0; j < VE; ++j) {
            if (v[j] >= l_min && order_key(v[j]) == cut_key && ++at == left) {
              const uint32_t idx = static_cast<uint32_t>(sl.first + (c0 + lane) * VE + j);
              for (int r = 0; r < C; ++r) *cluster.map_shared_rank(&S.cut_pos, r) = idx;
            }
          }
        }
        left -= __shfl_sync(0xffffffffu, incl, 31);
      }
    }
    cluster.sync();
    const int idx_cut = static_cast<int>(S.cut_pos);
    // the warps' sums of what is kept; everyone finds the draw's warp
    for (int c0 = sl.begin; c0 < sl.end; c0 += 32) {
      float v[VE];
      sl.get(c0 + lane, v);
#pragma unroll
      for (int j = 0; j < VE; ++j) {
        const uint32_t key = order_key(v[j]);
        const bool ok = v[j] >= l_min && (key > cut_key || (key == cut_key &&
                                          sl.first + (c0 + lane) * VE + j <= idx_cut));
        if (!__any_sync(0xffffffffu, ok)) continue;
        const unsigned long long w = weigh_call(weigh, ok ? v[j] : top);
        w_mine += ok ? w : 0;
      }
    }
    w_mine = warp_sum(w_mine);
    cut.key = cut_key;
    cut.idx = idx_cut;
  }
  if (generic || !list_on) {
    // every CTA finds the warp that the draw falls on
    if (lane < C) cluster.map_shared_rank(S.warp_mass, lane)[my_warp] = w_mine;
    cluster.sync();
    unsigned long long sum = 0, total = 0;
    for (int i = lane; i < warps; i += 32) {
      const unsigned long long w = S.warp_mass[i];
      total += w;
      if (i < my_warp) sum += w;
    }
    sum = warp_sum(sum);
    total = warp_sum(total);
    const unsigned long long to = target(total);
    if (!(sum <= to && to < sum + w_mine)) return;
    if (lane == 0) S.result = {1, my_warp, cut.key, cut.idx, sum, total, to};
    __syncwarp();
  }

  // ---- the warp that the draw falls on walks through its tokens
  const Result R = S.result;
  if (R.who != my_warp) return;
  unsigned long long before = R.before;
  for (int c0 = sl.begin; c0 < sl.end; c0 += 32) {
    float v[VE];
    sl.get(c0 + lane, v);
    unsigned long long w[VE], here = 0;
#pragma unroll
    for (int j = 0; j < VE; ++j) {
      const uint32_t key = order_key(v[j]);
      const bool ok = v[j] >= l_min && (key > R.cut_key || (key == R.cut_key &&
                                        sl.first + (c0 + lane) * VE + j <= R.idx_cut));
      w[j] = weigh(ok ? v[j] : top);
      if (!ok) w[j] = 0;
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
      if (sum <= R.to && R.to < sum + w[j]) {
        A.ids[row] = sl.first + (c0 + lane) * VE + j;
        if (A.probs) A.probs[row] = static_cast<float>(w[j]) / static_cast<float>(R.total);
      }
      sum += w[j];
    }
    before += __shfl_sync(0xffffffffu, incl, 31);
    if (before > R.to) break;
  }
}

template <typename LT>
static cudaError_t launch_sample(const SampArgs& a, int B, int cluster, cudaStream_t st) {
  const size_t smem = (static_cast<size_t>(a.slice) * sizeof(LT) + 31) / 16 * 16;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(sample_kernel<LT>), kMaxSlice, done);
  if (e != cudaSuccess) return e;
  return launch_cluster(sample_kernel<LT>, dim3(static_cast<unsigned>(B) * cluster),
                        dim3(kSampThreads), cluster, smem, st, a);
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
  // CTAs per row: enough that a slice is at most 64 KB (two CTAs per SM), and
  // more while the GPU is not full and a slice keeps 4 KB
  int cluster = 1;
  while (cluster < kMaxCluster && static_cast<long long>(V) * es > 65536ll * cluster) cluster *= 2;
  while (cluster < kMaxCluster && static_cast<long long>(B) * cluster < 152 &&
         static_cast<long long>(V) * es > 8192ll * cluster)
    cluster *= 2;
  SampArgs a = {logits, row_stride, u, temperature, top_k, top_p, min_p, ids, probs, V,
                (((V + cluster - 1) / cluster) + 7) / 8 * 8};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = logits_dtype == MOE_LOGITS_F32
                            ? launch_sample<float>(a, B, cluster, st)
                            : launch_sample<__nv_bfloat16>(a, B, cluster, st);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
