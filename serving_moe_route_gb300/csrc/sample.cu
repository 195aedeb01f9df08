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
//   A  the largest logit (and its lowest index: the answer of a greedy row)
//   B  with top-k or top-p: a histogram over bins of width t/64 below the
//      largest logit; counts for top-k, weights as well for top-p alone.  The
//      bin where the count or the weight passes its border bounds what is
//      kept.
//   C  if at most 512 tokens lie in the bins down to that one, they go to the
//      first CTA, whose threads rank them against each other (every thread
//      one token): top-k, top-p and the draw are sums over that list.
//   D  else the border is narrowed to a single logit value by histograms over
//      the bin's order keys (at most three), ties are counted in index order,
//      and the draw goes by the warps' sums over their slices.
// Rows without top-k and top-p go from A to D's draw.  Bound by the row's
// bytes for top-k, by the weights' instructions (about 40 a token) where the
// whole vocabulary has to be weighed.
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
constexpr int kBins = 2048;
constexpr int kList = kSampThreads;  // tokens that the list holds: one a thread
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
__constant__ unsigned long long kPow2[32] = {
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

// What turns a logit into a weight: the largest logit, log2(e) / t as a pair
// of floats, and this lane's entry of the table
struct Weigher {
  float top, ch, cl;
  uint32_t t_hi, t_lo;  // kPow2[lane] >> 13 and its low 13 bits

  // round(2^44 exp((l - top) / t)); every lane of the warp calls it.
  // x = (l - top) log2(e) / t as a pair ph + pl (both differences and
  // products with their rounding errors), x = k / 32 + r, 2^x = 2^(k >> 5)
  // T[k & 31] (1 + (2^r - 1)) with the bracket's main part in fixed point
  __device__ __forceinline__ unsigned long long operator()(float l) const {
    const float dh = l - top;
    const float b = dh - l;
    const float dl = (l - (dh - b)) - (top + b);
    const float ph = dh * ch;
    const bool live = ph > -46.0f;  // below, the weight rounds to 0
    const float pl = fmaf(dh, ch, -ph) + fmaf(dh, cl, dl * ch);
    const float kf = rintf((live ? ph : 0.0f) * 32.0f);
    const int k = static_cast<int>(kf);
    const float rh = fmaf(kf, -0.03125f, live ? ph : 0.0f);  // exact, |rh| <= 2^-6
    const int R = __float2int_rn(rh * 68719476736.0f);       // 2^36
    const float r2 = rh * rh;
    // pl ln 2, and the terms of degree 2 to 4 (with 2^pl's first order)
    float rest = fmaf(rh, 0.009618129107628477f, 0.05550410866482158f);
    rest = fmaf(rest, rh, 0.24022650695910072f);
    rest = fmaf(rest, r2, live ? pl * fmaf(rh, 0.4804530139182014f, 0.6931471805599453f) : 0.0f);
    const int E = static_cast<int>((static_cast<long long>(R) * 1488522236) >> 30) +
                  __float2int_rn(rest * 137438953472.0f);  // both in 2^-37
    const uint32_t hi = __shfl_sync(0xffffffffu, t_hi, k & 31);
    const uint32_t lo = __shfl_sync(0xffffffffu, t_lo, k & 31);
    const long long T = (static_cast<long long>(hi) << 13) | lo;
    const long long w = T + ((static_cast<long long>(hi) * E) >> 24);
    const int n = -(k >> 5);  // 0 .. 46
    const unsigned long long v =
        (((static_cast<unsigned long long>(w) << 1) >> n) + 1ull) >> 1;
    return live ? v : 0ull;
  }
};

// Values that the first CTA finds and all CTAs of the cluster read
struct Found {
  int bin;                    // bin where the border lies
  int count_above, count_in;  // tokens in better bins, in this one
  unsigned long long mass_above, mass_in, mass_all;
};

struct SampShared {
  uint32_t cnt[kBins], lo[kBins], hi[kBins];
  uint32_t list_key[kList];
  int list_idx[kList];
  unsigned long long list_w[kList];
  unsigned long long best[kMaxCluster];                // written by every CTA of the cluster
  unsigned long long warp_mass[kMaxCluster * kSampWarps];  // likewise
  int warp_ties[kMaxCluster * kSampWarps];             // likewise
  uint32_t key_lo[kMaxCluster], key_hi[kMaxCluster];   // likewise
  int idx_cut;                                         // likewise
  int list_n;
  Found found;
  long long scan[2 * kSampWarps];
  float ch, cl, l_min, u, p;
  double d_min;
  int k;
  float t;
  int min_on;
};

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
__global__ void __launch_bounds__(kSampThreads) sample_kernel(const SampArgs A) {
  constexpr int VE = Slice<LT>::VE;
  constexpr int ES = sizeof(LT);
  extern __shared__ __align__(16) uint8_t slice_smem[];
  __shared__ SampShared S;
  cg::cluster_group cluster = cg::this_cluster();
  const int C = static_cast<int>(cluster.num_blocks());
  const int rank = static_cast<int>(cluster.block_rank());
  const int row = blockIdx.x / C;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool lead = rank == 0;
  pdl_wait();

  // ---- the slice: 16-byte chunks of the row; the elements of the first and
  // the last chunk that lie outside the slice become -inf
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
  for (int c = tid; c < sl.chunks; c += kSampThreads) {
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
    if (t > 0.0f) {
      double c = 1.4426950408889634074 / static_cast<double>(t);
      c = fmin(c, 1e30);
      S.ch = static_cast<float>(c);
      S.cl = static_cast<float>(c - S.ch);
      S.min_on = m > 0.0f;
      S.d_min = m > 0.0f ? static_cast<double>(t) * log(fmin(static_cast<double>(m), 1.0)) : 0.0;
    }
    S.list_n = 0;
  }
  for (int i = tid; i < kBins; i += kSampThreads) S.cnt[i] = S.lo[i] = S.hi[i] = 0;
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncthreads();

  // ---- A: the largest logit; NaN becomes -inf and +inf the largest float
  unsigned long long best = 0;
  for (int c = sl.begin + lane; c < sl.end; c += 32) {
    float v[VE];
    sl.get(c, v);
#pragma unroll
    for (int j = 0; j < VE; ++j) {
      if (!(v[j] < INFINITY)) {
        v[j] = v[j] != v[j] ? -INFINITY : FLT_MAX;
        LT* x = reinterpret_cast<LT*>(slice_smem) + c * VE + j;
        // bf16 has no FLT_MAX; its +inf stays and is read as FLT_MAX by order
        if constexpr (ES == 4) *x = v[j];
        else if (v[j] < 0) *x = __ushort_as_bfloat16(0xff80);
        else *x = __ushort_as_bfloat16(0x7f7f);
        if constexpr (ES == 2) {
          if (v[j] > 0) v[j] = __bfloat162float(*x);
        }
      }
      if (v[j] > -INFINITY) {
        const unsigned long long cand = (static_cast<unsigned long long>(order_key(v[j])) << 32) |
                                        (0xffffffffu - static_cast<uint32_t>(sl.first + c * VE + j));
        best = max(best, cand);
      }
    }
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1)
    best = max(best, __shfl_xor_sync(0xffffffffu, best, off));
  if (lane == 0) S.scan[warp] = static_cast<long long>(best);
  __syncthreads();
  if (tid < C) {
    for (int w = 0; w < kSampWarps; ++w)
      best = max(best, static_cast<unsigned long long>(S.scan[w]));
    cluster.map_shared_rank(S.best, tid)[rank] = best;
  }
  cluster.sync();
  best = 0;
  for (int r = 0; r < C; ++r) best = max(best, S.best[r]);
  if (best == 0 || !(S.t > 0.0f)) {  // nothing to draw, or greedy
    if (lead && tid == 0) {
      A.ids[row] = best == 0 ? -1 : static_cast<int>(0xffffffffu - static_cast<uint32_t>(best));
      if (A.probs) A.probs[row] = best == 0 ? 0.0f : 1.0f;
    }
    cluster.sync();  // no CTA leaves while another writes into it
    return;
  }
  const uint32_t top_key = static_cast<uint32_t>(best >> 32);
  Weigher weigh;
  weigh.top = key_value(top_key);
  weigh.ch = S.ch;
  weigh.cl = S.cl;
  weigh.t_hi = static_cast<uint32_t>(kPow2[lane] >> 13);
  weigh.t_lo = static_cast<uint32_t>(kPow2[lane] & 8191);
  if (tid == 0) {
    // the smallest logit that min-p keeps: exact tests around its estimate
    float lm = -FLT_MAX;
    if (S.min_on) {
      const double top = weigh.top, d = S.d_min;
      lm = fminf(weigh.top, fmaxf(-FLT_MAX, static_cast<float>(top + d)));
      for (int i = 0; i < 4 && lm > -FLT_MAX; ++i) {
        const float below = key_value(order_key(lm) - 1);
        if (!(static_cast<double>(below) - top >= d)) break;
        lm = below;
      }
      for (int i = 0; i < 4 && lm < weigh.top; ++i) {
        if (static_cast<double>(lm) - top >= d) break;
        lm = key_value(order_key(lm) + 1);
      }
    }
    S.l_min = lm;
  }
  __syncthreads();
  const float l_min = S.l_min;
  const int k = S.k;
  const bool p_on = S.p < 1.0f;
  const float bin_scale = fminf(64.0f / S.t, 1e30f);
  auto bin_of = [&](float l) {
    return min(kBins - 1, static_cast<int>((weigh.top - l) * bin_scale));
  };

  // A histogram of the tokens that `in` takes, by bin `of`: counts, and
  // weights if `mass`.  The last bin collects the far tail: its sums are kept
  // per thread and added once.
  auto histogram = [&](bool mass, auto in, auto of) {
    unsigned tail_n = 0;
    unsigned long long tail_w = 0;
    for (int c0 = sl.begin; c0 < sl.end; c0 += 32) {
      float v[VE];
      sl.get(c0 + lane, v);
#pragma unroll
      for (int j = 0; j < VE; ++j) {
        const bool ok = v[j] >= l_min && in(v[j]);
        unsigned long long w = 0;
        if (mass) w = weigh(ok ? v[j] : weigh.top);
        if (ok) {
          const int b = of(v[j]);
          if (b == kBins - 1) {
            ++tail_n;
            tail_w += w;
          } else {
            atomicAdd(&S.cnt[b], 1u);
            if (mass && w) {
              const uint32_t add = static_cast<uint32_t>(w);
              const uint32_t old = atomicAdd(&S.lo[b], add);
              const uint32_t up = static_cast<uint32_t>(w >> 32) + (old + add < old ? 1u : 0u);
              if (up) atomicAdd(&S.hi[b], up);
            }
          }
        }
      }
    }
    tail_n = __reduce_add_sync(0xffffffffu, tail_n);
    tail_w = warp_sum(tail_w);
    if (lane == 0 && tail_n) {
      atomicAdd(&S.cnt[kBins - 1], tail_n);
      const uint32_t add = static_cast<uint32_t>(tail_w);
      const uint32_t old = atomicAdd(&S.lo[kBins - 1], add);
      atomicAdd(&S.hi[kBins - 1],
                static_cast<uint32_t>(tail_w >> 32) + (old + add < old ? 1u : 0u));
    }
  };
  // The bin where the count passes `need_n`, or the weight its border, on top
  // of what lies above this histogram; to every CTA.  need_p > 0: the border
  // is that share of the histogram's weight.  Clears the histogram.
  auto find = [&](bool mass, int need_n, unsigned long long need_w, float need_p, int above_n,
                  unsigned long long above_w) {
    cluster.sync();
    if (lead) {
      constexpr int PER = kBins / kSampThreads;
      long long cn[PER], cw[PER], sn = 0, sw = 0;
#pragma unroll
      for (int i = 0; i < PER; ++i) cn[i] = cw[i] = 0;
      for (int r = 0; r < C; ++r) {
        const SampShared* o = cluster.map_shared_rank(&S, r);
        const uint4 a = *reinterpret_cast<const uint4*>(&o->cnt[tid * PER]);
        cn[0] += a.x; cn[1] += a.y; cn[2] += a.z; cn[3] += a.w;
        if (mass) {
          const uint4 l = *reinterpret_cast<const uint4*>(&o->lo[tid * PER]);
          const uint4 h = *reinterpret_cast<const uint4*>(&o->hi[tid * PER]);
          cw[0] += (static_cast<long long>(h.x) << 32) + l.x;
          cw[1] += (static_cast<long long>(h.y) << 32) + l.y;
          cw[2] += (static_cast<long long>(h.z) << 32) + l.z;
          cw[3] += (static_cast<long long>(h.w) << 32) + l.w;
        }
      }
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        sn += cn[i];
        sw += cw[i];
      }
      long long en, ew, tn, tw;
      scan_pair(sn, sw, S.scan, en, ew, tn, tw);
      if (need_p > 0.0f)
        need_w = static_cast<unsigned long long>(
            ceil(static_cast<double>(need_p) * static_cast<double>(tw)));
      need_w = max(need_w, 1ull);
      if (tid == 0) {  // the border lies past everything: the last bin, all of it
        S.found.bin = kBins - 1;
        S.found.count_above = static_cast<int>(above_n + tn);
        S.found.mass_above = above_w + tw;
        S.found.count_in = 0;
        S.found.mass_in = 0;
      }
      __syncthreads();
      long long n_at = above_n + en, w_at = static_cast<long long>(above_w) + ew;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const bool here = mass ? w_at < static_cast<long long>(need_w) &&
                                     w_at + cw[i] >= static_cast<long long>(need_w)
                               : n_at < need_n && n_at + cn[i] >= need_n;
        if (here) {
          S.found.bin = tid * PER + i;
          S.found.count_above = static_cast<int>(n_at);
          S.found.count_in = static_cast<int>(cn[i]);
          S.found.mass_above = static_cast<unsigned long long>(w_at);
          S.found.mass_in = static_cast<unsigned long long>(cw[i]);
        }
        n_at += cn[i];
        w_at += cw[i];
      }
      if (tid == 0) S.found.mass_all = static_cast<unsigned long long>(above_w + tw);
    }
    cluster.sync();
    const Found f = *cluster.map_shared_rank(&S.found, 0);
    for (int i = tid; i < kBins; i += kSampThreads) S.cnt[i] = S.lo[i] = S.hi[i] = 0;
    cluster.sync();
    return f;
  };

  auto all = [](float) { return true; };
  const double u = S.u > 0.0f ? static_cast<double>(S.u) : 0.0;
  // the first running sum above u * total is above this whole number
  auto target = [&](unsigned long long total) {
    const double t = u * static_cast<double>(total);
    const unsigned long long i = t >= 9.2e18 ? ~0ull : static_cast<unsigned long long>(t);
    return min(i, total - 1);
  };

  uint32_t cut_key = 0;    // kept: order key above it,
  int cut_ties = INT_MAX;  // and so many, by index, of those equal to it
  int ties_in = 0;         // how many there are
  if (k || p_on) {
    // ---- B
    const bool by_mass = !k;
    histogram(by_mass, all, bin_of);
    Found f = find(by_mass, k, 0, by_mass ? fmaxf(S.p, 1e-30f) : 0.0f, 0, 0);
    const bool bound = f.count_in > 0;  // else top-k keeps everything
    if (f.count_above + f.count_in <= kList) {
      // ---- C: the tokens of the bins down to f.bin, to the first CTA
      for (int c0 = sl.begin; c0 < sl.end; c0 += 32) {
        float v[VE];
        sl.get(c0 + lane, v);
#pragma unroll
        for (int j = 0; j < VE; ++j) {
          if (v[j] >= l_min && bin_of(v[j]) <= f.bin) {
            const int at = atomicAdd(&S.list_n, 1);
            S.list_key[at] = order_key(v[j]);
            S.list_idx[at] = sl.first + (c0 + lane) * VE + j;
          }
        }
      }
      cluster.sync();
      if (lead) {
        int n_list = S.list_n;
        for (int r = 1; r < C; ++r) {
          const SampShared* o = cluster.map_shared_rank(&S, r);
          const int m = o->list_n;
          if (tid < m) {
            S.list_key[n_list + tid] = o->list_key[tid];
            S.list_idx[n_list + tid] = o->list_idx[tid];
          }
          n_list += m;
        }
        __syncthreads();
        const bool mine = tid < n_list;
        const uint32_t key = mine ? S.list_key[tid] : top_key;
        const int idx = mine ? S.list_idx[tid] : INT_MAX;
        const unsigned long long w = weigh(key_value(key));
        S.list_w[tid] = mine ? w : 0;
        __syncthreads();
        int better = 0;
        unsigned long long before = 0;
        for (int j = 0; j < n_list; ++j) {
          const uint32_t kj = S.list_key[j];
          if (kj > key || (kj == key && S.list_idx[j] < idx)) {
            ++better;
            before += S.list_w[j];
          }
        }
        bool keep = mine && (!k || better < k);
        long long ex, unused, mass, tot;
        scan_pair(keep ? static_cast<long long>(w) : 0, 0, S.scan, ex, unused, mass, tot);
        if (p_on) {
          // without top-k the share is of the whole vocabulary's weight
          const double all_w = k ? static_cast<double>(mass) : static_cast<double>(f.mass_all);
          const unsigned long long border =
              static_cast<unsigned long long>(ceil(static_cast<double>(fmaxf(S.p, 0.0f)) * all_w));
          keep = keep && (better == 0 || before < border);
          scan_pair(keep ? static_cast<long long>(w) : 0, 0, S.scan, ex, unused, mass, tot);
        }
        __syncthreads();
        S.list_w[tid] = keep ? w : 0;
        __syncthreads();
        const unsigned long long to = target(static_cast<unsigned long long>(mass));
        unsigned long long sum = 0;
        for (int j = 0; j < n_list; ++j)
          if (S.list_idx[j] < idx) sum += S.list_w[j];
        if (keep && w && sum <= to && to < sum + w) {
          A.ids[row] = idx;
          if (A.probs)
            A.probs[row] = static_cast<float>(w) / static_cast<float>(mass);
        }
      }
      cluster.sync();
      return;
    }
    // ---- D: narrow the border down to one value.  `floor_key`: keys below
    // it are out already (top-k's cut, while top-p's is looked for)
    auto narrow = [&](bool mass, int need_n, unsigned long long need_w, uint32_t floor_key,
                      Found& g) {
      uint32_t lo = 0xffffffffu, hi = 0;
      for (int c0 = sl.begin; c0 < sl.end; c0 += 32) {
        float v[VE];
        sl.get(c0 + lane, v);
#pragma unroll
        for (int j = 0; j < VE; ++j)
          if (v[j] >= l_min && bin_of(v[j]) == g.bin && order_key(v[j]) >= floor_key) {
            lo = min(lo, order_key(v[j]));
            hi = max(hi, order_key(v[j]));
          }
      }
      lo = __reduce_min_sync(0xffffffffu, lo);
      hi = __reduce_max_sync(0xffffffffu, hi);
      if (lane == 0) S.scan[warp] = (static_cast<long long>(hi) << 32) | lo;
      __syncthreads();
      if (tid < C) {
        for (int w = 0; w < kSampWarps; ++w) {
          lo = min(lo, static_cast<uint32_t>(S.scan[w]));
          hi = max(hi, static_cast<uint32_t>(static_cast<unsigned long long>(S.scan[w]) >> 32));
        }
        cluster.map_shared_rank(S.key_lo, tid)[rank] = lo;
        cluster.map_shared_rank(S.key_hi, tid)[rank] = hi;
      }
      cluster.sync();
      lo = 0xffffffffu;
      hi = 0;
      for (int r = 0; r < C; ++r) {
        lo = min(lo, S.key_lo[r]);
        hi = max(hi, S.key_hi[r]);
      }
      for (;;) {
        const uint32_t width = hi - lo;
        const int sh = max(0, 32 - __clz(width) - 11);  // 2^11 bins
        histogram(mass,
                  [&](float x) {
                    const uint32_t key = order_key(x);
                    return key >= lo && key <= hi;
                  },
                  [&](float x) { return static_cast<int>((hi - order_key(x)) >> sh); });
        g = find(mass, need_n, need_w, 0.0f, g.count_above, g.mass_above);
        hi -= static_cast<uint32_t>(g.bin) << sh;
        if (sh == 0) break;
        lo = max(lo, hi - ((1u << sh) - 1u));
      }
      return hi;
    };
    unsigned long long need_w = 0;
    if (k && bound) {
      cut_key = narrow(false, k, 0, 0, f);
      cut_ties = k - f.count_above;
      ties_in = f.count_in;
    }
    if (p_on) {
      unsigned long long floor_w = 0;  // weight of one token at top-k's cut
      if (k) {
        // the weight that top-k left: of the keys above its cut, and its ties
        const uint32_t floor_key = cut_key;
        histogram(true, [&](float x) { return order_key(x) > floor_key; }, bin_of);
        f = find(true, 0, ~0ull >> 1, 0.0f, 0, 0);
        floor_w = cut_ties == INT_MAX ? 0 : weigh(key_value(cut_key));
        const unsigned long long left =
            f.mass_all + (cut_ties == INT_MAX ? 0 : floor_w * static_cast<unsigned long long>(cut_ties));
        need_w = max(1ull, static_cast<unsigned long long>(
                               ceil(static_cast<double>(fmaxf(S.p, 0.0f)) *
                                    static_cast<double>(left))));
        if (need_w <= f.mass_all) {  // else the border lies among top-k's ties
          histogram(true, [&](float x) { return order_key(x) > floor_key; }, bin_of);
          f = find(true, 0, need_w, 0.0f, 0, 0);
          cut_key = narrow(true, 0, need_w, floor_key + 1, f);
          const unsigned long long w = weigh(key_value(cut_key));
          cut_ties = static_cast<int>((need_w - f.mass_above + w - 1) / w);
          ties_in = f.count_in;
        } else {
          cut_ties = min(static_cast<unsigned long long>(cut_ties),
                         (need_w - f.mass_all + floor_w - 1) / floor_w);
        }
      } else {
        need_w = max(1ull, static_cast<unsigned long long>(
                               ceil(static_cast<double>(fmaxf(S.p, 1e-30f)) *
                                    static_cast<double>(f.mass_all))));
        cut_key = narrow(true, 0, need_w, 0, f);
        const unsigned long long w = weigh(key_value(cut_key));
        cut_ties = static_cast<int>((need_w - f.mass_above + w - 1) / w);
        ties_in = f.count_in;
      }
    }
  }

  // ---- the index of the last kept tie, where not all are kept
  int idx_cut = INT_MAX;
  if (cut_ties < ties_in) {
    int mine = 0;
    for (int c0 = sl.begin; c0 < sl.end; c0 += 32) {
      float v[VE];
      sl.get(c0 + lane, v);
#pragma unroll
      for (int j = 0; j < VE; ++j) mine += v[j] >= l_min && order_key(v[j]) == cut_key;
    }
    mine = __reduce_add_sync(0xffffffffu, mine);
    if (lane < C) cluster.map_shared_rank(S.warp_ties, lane)[rank * kSampWarps + warp] = mine;
    cluster.sync();
    int before = 0;
    for (int i = lane; i < rank * kSampWarps + warp; i += 32) before += S.warp_ties[i];
    before = __reduce_add_sync(0xffffffffu, before);
    if (before < cut_ties && before + mine >= cut_ties) {
      int left = cut_ties - before;  // the left-th tie of this warp
      for (int c0 = sl.begin; c0 < sl.end && left > 0; c0 += 32) {
        float v[VE];
        sl.get(c0 + lane, v);
        int here = 0;
#pragma unroll
        for (int j = 0; j < VE; ++j) here += v[j] >= l_min && order_key(v[j]) == cut_key;
        int incl = here;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, incl, off);
          if (lane >= off) incl += y;
        }
        if (incl >= left && incl - here < left) {
          int at = incl - here;
#pragma unroll
          for (int j = 0; j < VE; ++j) {
            if (v[j] >= l_min && order_key(v[j]) == cut_key && ++at == left) {
              const int idx = sl.first + (c0 + lane) * VE + j;
              for (int r = 0; r < C; ++r) *cluster.map_shared_rank(&S.idx_cut, r) = idx;
            }
          }
        }
        left -= __shfl_sync(0xffffffffu, incl, 31);
      }
    }
    cluster.sync();
    idx_cut = S.idx_cut;
  }

  // ---- the draw: the warps' sums, then the one warp whose slice it falls in
  auto kept = [&](float x, int idx) {
    const uint32_t key = order_key(x);
    return x >= l_min && (key > cut_key || (key == cut_key && idx <= idx_cut));
  };
  unsigned long long mine = 0;
  for (int c0 = sl.begin; c0 < sl.end; c0 += 32) {
    float v[VE];
    sl.get(c0 + lane, v);
#pragma unroll
    for (int j = 0; j < VE; ++j) {
      const bool ok = kept(v[j], sl.first + (c0 + lane) * VE + j);
      const unsigned long long w = weigh(ok ? v[j] : weigh.top);
      mine += ok ? w : 0;
    }
  }
  mine = warp_sum(mine);
  if (lane < C) cluster.map_shared_rank(S.warp_mass, lane)[rank * kSampWarps + warp] = mine;
  cluster.sync();
  unsigned long long before = 0, total = 0;
  for (int i = lane; i < C * kSampWarps; i += 32) {
    const unsigned long long w = S.warp_mass[i];
    total += w;
    if (i < rank * kSampWarps + warp) before += w;
  }
  before = warp_sum(before);
  total = warp_sum(total);
  const unsigned long long to = target(total);
  if (before <= to && to < before + mine) {
    for (int c0 = sl.begin; c0 < sl.end; c0 += 32) {
      float v[VE];
      sl.get(c0 + lane, v);
      unsigned long long w[VE], here = 0;
#pragma unroll
      for (int j = 0; j < VE; ++j) {
        const bool ok = kept(v[j], sl.first + (c0 + lane) * VE + j);
        w[j] = weigh(ok ? v[j] : weigh.top);
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
        if (sum <= to && to < sum + w[j]) {
          A.ids[row] = sl.first + (c0 + lane) * VE + j;
          if (A.probs) A.probs[row] = static_cast<float>(w[j]) / static_cast<float>(total);
        }
        sum += w[j];
      }
      before += __shfl_sync(0xffffffffu, incl, 31);
      if (before > to) break;
    }
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
