// attn_tree.cuh -- what the kernels of moe_attn_tree share: the arguments, the
// deal of the work to CTAs, and which tokens a row attends.
//
// A unit is (request, kv head, block of ROWS rows), a row being (node, query head
// of that kv head), nodes in order.  Its tokens form tiles of TILE; it counts its
// tiles and END more for its end.  CTAs work in groups of as many as the largest
// request has blocks (8 at most), one block each, on the same tokens at the same
// time, so that all but one find them in L2; a request of fewer blocks leaves the
// rest of the group idle.  The counts of all (request, kv head), in order, are cut
// into equal contiguous ranges, one per group of a single wave, so that ragged
// lengths and one long request balance alike.  A range may begin and end inside a
// unit; the unit's parts go to the workspace and a second kernel joins them in order.
#pragma once
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

struct TreeArgs {
  const char *k, *v;
  long long s_page, s_token, s_head;  // bytes
  const float *k_scale, *v_scale;
  const void* q;
  long long q_n, q_h;  // elements
  void* out;
  long long o_n, o_h;  // elements
  float* lse;
  const int* table;
  long long table_stride;
  const int *starts, *lens;
  const unsigned long long* masks;
  float* part_o;    // [2 * ctas][ROWS][DP]
  float2* part_ml;  // [2 * ctas][ROWS]
  int4* info;       // [ctas] {unit's request, unit in request, parts, place + 2^16 group}
  unsigned* err;
  float scale_log2;
  int N, B, Hq, heads, group, words, max_new;
  int dim, page, page_shift, num_pages, max_pages, window;
  int box;  // tokens that TMA brings at a time; 0: it cannot
};

// A request's rows and tokens
struct TreeSpan {
  int row0, n, use;  // first row, rows, rows that are worked on
  int ctx, first, len;  // context tokens, where tiles begin, end
};

__device__ __forceinline__ TreeSpan tree_span(const TreeArgs& A, int r, bool& cut) {
  TreeSpan s;
  s.row0 = max(0, min(A.starts[r], A.N));
  s.n = max(s.row0, min(A.starts[r + 1], A.N)) - s.row0;
  s.use = min(s.n, A.max_new);
  const int all = max(A.lens[r], 0);
  const long long room = static_cast<long long>(A.max_pages) * A.page;
  s.len = static_cast<int>(min(static_cast<long long>(all), room));
  s.ctx = max(0, all - s.n);
  // (tiles begin at multiples of their size, as TMA's boxes must)
  s.first = A.window > 0 ? min(max(0, s.ctx - A.window), s.len) & ~127 : 0;
  if (s.n > 0 && (s.use < s.n || s.len < all)) cut = true;
  return s;
}
// 16 bytes to shared memory; zeros, and nothing is read, where they are not real
__device__ __forceinline__ void tree_cp16(uint32_t dst, const void* src, bool real) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(real ? 16 : 0)
               : "memory");
}
constexpr int kTreeGroup = 8;  // CTAs of a group at most

// blocks of a request's rows
template <int ROWS>
__device__ __forceinline__ int tree_blocks(const TreeArgs& A, const TreeSpan& s) {
  return (s.use * A.group + ROWS - 1) / ROWS;
}
template <int TILE>
__device__ __forceinline__ int tree_tiles(const TreeSpan& s) {
  return max(1, (s.len - s.first + TILE - 1) / TILE);
}

// Where this CTA's range begins, in shared memory
struct TreeStart {
  long long left, end, total;
  int b, x, t, groups;
  int size, place;  // CTAs of a group, this one's place in it
};

// A CTA's range, walked part by part: tiles [t0, t1) of the nt of unit x (kv head
// and round) of request b, this CTA's block of it.  Every role of a CTA keeps one.
template <int ROWS, int TILE, int END>
struct TreeWalk {
  TreeSpan s;
  int b, x, t, nt, rounds, blocks;
  long long left, end;  // places from here on; the range's end, counted over all units
  int t0, t1, size, place;

  __device__ __forceinline__ int head() const { return x / rounds; }
  __device__ __forceinline__ int block() const { return x % rounds * size + place; }
  __device__ __forceinline__ void enter(const TreeArgs& A, int request) {
    bool cut = false;
    for (b = request; b < A.B; ++b) {
      s = tree_span(A, b, cut);
      blocks = tree_blocks<ROWS>(A, s);
      if (blocks > 0) break;
    }
    rounds = (blocks + size - 1) / size;
    nt = tree_tiles<TILE>(s);
    x = 0;
    t = 0;
  }
  __device__ __forceinline__ void skip(const TreeArgs& A) {
    t = 0;
    if (left > 0 && ++x >= rounds * A.heads) enter(A, b + 1);
  }
  // the next part; false at the range's end.  `at` is its unit
  __device__ __forceinline__ bool next(const TreeArgs& A, TreeWalk& at) {
    while (left > 0) {
      at = *this;
      at.t0 = t;
      at.t1 = static_cast<int>(min(static_cast<long long>(nt), t + left));
      left -= at.t1 - t;
      if (at.t1 < nt) {
        left = 0;
      } else {
        left -= END;
        skip(A);
      }
      if (at.block() < at.blocks) return true;  // else there is none for this CTA
    }
    return false;
  }
};

// Every thread of the CTA (a multiple of 32, at most 1024) calls it; out and sums
// (33 of them) are in shared memory
template <int ROWS, int TILE, int END>
__device__ __forceinline__ void tree_begin(const TreeArgs& A, TreeStart* out, long long* sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int threads = blockDim.x, nw = threads >> 5;
  bool cut = false;
  const int per = (A.B - 1) / threads + 1;
  const int b0 = static_cast<int>(min(static_cast<long long>(A.B),
                                      static_cast<long long>(threadIdx.x) * per));
  const int b1 = b0 + min(per, A.B - b0);
  // the size of a group: the most blocks that a request has
  TreeSpan s;
  int most = 0;
  for (int b = b0; b < b1; ++b) {
    s = tree_span(A, b, cut);
    most = max(most, tree_blocks<ROWS>(A, s));
  }
  most = __reduce_max_sync(0xffffffffu, most);
  if (lane == 0) sums[warp] = most;
  __syncthreads();
  for (int w = 0; w < nw; ++w) most = max(most, static_cast<int>(sums[w]));
  const int size = max(1, min(min(most, kTreeGroup), static_cast<int>(gridDim.x)));
  __syncthreads();
  auto places = [&](const TreeSpan& s) {
    return static_cast<long long>((tree_blocks<ROWS>(A, s) + size - 1) / size) * A.heads *
           (tree_tiles<TILE>(s) + END);
  };
  long long mine = 0;
  for (int b = b0; b < b1; ++b) {
    if (per > 1) s = tree_span(A, b, cut);
    mine += places(s);
  }
  long long incl = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += y;
  }
  if (lane == 31) sums[warp] = incl;
  __syncthreads();
  long long before = 0, total = 0;
  for (int w = 0; w < nw; ++w) {
    if (w < warp) before += sums[w];
    total += sums[w];
  }
  if (cut && A.err && blockIdx.x == 0) atomicOr(A.err, MOE_DEVERR_NO_SPACE);
  const int groups = static_cast<int>(min(static_cast<long long>(gridDim.x / size), total));
  const int g = blockIdx.x / size;
  if (threadIdx.x == 0) {
    A.info[blockIdx.x] = make_int4(0, 0, 0, 0);
    out->groups = groups;
    out->size = size;
    out->place = blockIdx.x % size;
    out->total = total;
    if (g >= groups) out->left = 0;
  }
  if (g < groups) {
    const long long begin = g * total / groups, end = (g + 1) * total / groups;
    const long long lo = before + incl - mine, hi = before + incl;
    if (begin >= lo && begin < hi) {
      long long at = lo;
      int b = b0;
      for (; per > 1; ++b) {
        s = tree_span(A, b, cut);
        const long long n = places(s);
        if (begin < at + n) break;
        at += n;
      }
      const int one = tree_tiles<TILE>(s) + END;
      out->b = b;
      out->x = static_cast<int>((begin - at) / one);
      out->t = static_cast<int>(begin - at - static_cast<long long>(out->x) * one);
      out->left = end - begin;
      out->end = end;
    }
  }
  __syncthreads();
}
template <int ROWS, int TILE, int END>
__device__ __forceinline__ TreeWalk<ROWS, TILE, END> tree_walk(const TreeArgs& A,
                                                               const TreeStart& w) {
  TreeWalk<ROWS, TILE, END> k;
  k.left = w.left;
  k.end = w.end;
  k.size = w.size;
  k.place = w.place;
  if (k.left <= 0) return k;
  k.enter(A, w.b);
  k.x = w.x;
  k.t = w.t;
  if (k.t >= k.nt) {  // the range begins with a unit's end: on to the next
    k.left -= k.nt + END - k.t;
    k.skip(A);
  }
  return k;
}

// The record of a unit that goes on behind this CTA's range (one thread)
template <int ROWS, int TILE, int END>
__device__ __forceinline__ void tree_record(const TreeArgs& A, const TreeStart& w,
                                            const TreeWalk<ROWS, TILE, END>& at) {
  // at: as `next` left it, its `left` counted from t0 on
  const long long from = at.end - at.left - at.t0, to = from + at.nt - 1;
  const int g0 = static_cast<int>(((from + 1) * w.groups - 1) / w.total);
  const int g1 = static_cast<int>(((to + 1) * w.groups - 1) / w.total);
  const int mine = static_cast<int>(blockIdx.x) / w.size;
  A.info[blockIdx.x] = make_int4(at.b, at.x, g1 - g0 + 1, (mine - g0) | w.size << 16);
}

// ------------------------------------------------------------ what a row attends
// A node's mask, in registers
struct TreeMask {
  unsigned long long m[MOE_TREE_MAX / 64];
};
__device__ __forceinline__ TreeMask tree_mask(const TreeArgs& A, const TreeSpan& s, int i) {
  TreeMask t;
#pragma unroll
  for (int w = 0; w < MOE_TREE_MAX / 64; ++w) {
    if (A.masks) {
      t.m[w] = w < A.words
                   ? __ldg(A.masks + static_cast<long long>(s.row0 + i) * A.words + w)
                   : 0;
    } else {  // nodes up to i
      const int n = i + 1 - 64 * w;
      t.m[w] = n <= 0 ? 0 : n >= 64 ? ~0ull : (1ull << n) - 1;
    }
  }
  return t;
}
// 32 bits of it from new token j on (j may be negative), of the tokens there are
__device__ __forceinline__ uint32_t tree_bits(const TreeSpan& s, const TreeMask& t, int j) {
  const int lim = min(s.n, s.len - s.ctx);
  if (j >= lim || j <= -32) return 0;
  uint32_t bits;
  if (j < 0) {
    bits = static_cast<uint32_t>(t.m[0]) << -j;
  } else {
    const int w = j >> 6, sh = j & 63;
    unsigned long long lo = 0, hi = 0;
#pragma unroll
    for (int k = 0; k < MOE_TREE_MAX / 64; ++k) {
      if (w == k) lo = t.m[k];
      if (w + 1 == k) hi = t.m[k];
    }
    bits = static_cast<uint32_t>(lo >> sh);
    if (sh > 32) bits |= static_cast<uint32_t>(hi << (64 - sh));
  }
  if (lim - j < 32) bits &= (1u << (lim - j)) - 1;
  return bits;
}
// first token that node i, whose mask t is, attends: of more new tokens than the window
// the highest count, which for a path from the root are the last
__device__ __forceinline__ int tree_low(const TreeArgs& A, const TreeSpan& s, const TreeMask& t,
                                        int i) {
  if (A.window <= 0) return 0;
  const int lim = min(s.n, s.len - s.ctx);
  int c = 0;
#pragma unroll
  for (int w = 0; w < MOE_TREE_MAX / 64; ++w) {
    const int k = lim - 64 * w;
    c += __popcll(k <= 0 ? 0 : k >= 64 ? t.m[w] : t.m[w] & ((1ull << k) - 1));
  }
  int low = max(0, s.ctx + c - A.window);
  if (c > A.window && A.masks) {  // (a short program: the mask is read again)
    low = s.ctx;
    int extra = c - A.window;
#pragma unroll 1
    for (int w = 0; extra > 0; ++w) {
      unsigned long long m = __ldg(A.masks + static_cast<long long>(s.row0 + i) * A.words + w);
#pragma unroll 1
      for (; extra > 0 && m; --extra, m &= m - 1)
        low = s.ctx + 64 * w + __ffsll(static_cast<long long>(m));
    }
  }
  return low;
}
// which of the 32 tokens from pos on its node attends (by its mask and window alone)
__device__ __forceinline__ uint32_t tree_attends(const TreeSpan& s, const TreeMask& t, int low,
                                                 int pos) {
  const int end = min(s.ctx, s.len);
  uint32_t bits = pos >= end ? 0 : end - pos < 32 ? (1u << (end - pos)) - 1 : ~0u;
  bits |= tree_bits(s, t, pos - s.ctx);
  return low <= pos ? bits : low - pos < 32 ? bits & (~0u << (low - pos)) : 0;
}

__device__ __forceinline__ float tree_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// weights of e4m3 caches, which are f16, are lifted by 2^kTreeLift
constexpr float kTreeLift = 13.0f;
// ln(sum 2^top): top without the lift and sum without it are both near what their
// rounding should be relative to
template <int KV>
__device__ __forceinline__ float tree_lse(float top, float sum) {
  constexpr float lift = KV == MOE_KV_E4M3 ? kTreeLift : 0.0f;
  if (top == -INFINITY) return -INFINITY;
  return ((top + lift) + log2f(sum * exp2f(-lift))) * 0.6931471805599453f;
}
__device__ __forceinline__ uint32_t tree_bf16x2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
template <int KV>
__device__ __forceinline__ void tree_store4(void* out, long long at, float a, float b, float c,
                                            float d) {
  if constexpr (KV == MOE_KV_F32)
    *reinterpret_cast<float4*>(static_cast<float*>(out) + at) = make_float4(a, b, c, d);
  else
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(out) + at) =
        make_uint2(tree_bf16x2(a, b), tree_bf16x2(c, d));
}

// Joins the parts of the units that range borders cut.  A unit that begins in CTA
// c and does not end there has c's first slot, then the second slots of the CTAs
// at its place in the next groups.  The kTreeJoinBlocks blocks of each CTA that it
// does not end in deal its rows out, a row a warp.  A few parts at a time are loaded
// along with their maxima and rescaled to the warp's reference so far, in order.
constexpr int kTreeJoinWarps = 8, kTreeJoinBlocks = 4;
template <int KV, int DP, int ROWS>
__global__ void __launch_bounds__(32 * kTreeJoinWarps)
    tree_join_kernel(const __grid_constant__ TreeArgs A) {
  constexpr int VL = DP / 32;  // columns per lane
  constexpr int kTreeAhead = 4;
  pdl_wait();
  const int4 unit = A.info[blockIdx.x];
  const int parts = unit.z, place = unit.w & 0xffff, size = unit.w >> 16;
  if (parts == 0) return;
  const int cta = blockIdx.x - place * size;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  bool cut = false;
  const TreeSpan s = tree_span(A, unit.x, cut);
  const int rounds = (tree_blocks<ROWS>(A, s) + size - 1) / size;
  const int kvh = unit.y / rounds, r0 = (unit.y % rounds * size + cta % size) * ROWS;
  const int rows = min(ROWS, s.use * A.group - r0);
  const float mul = KV == MOE_KV_E4M3 ? A.v_scale[kvh] : 1.0f;
#pragma unroll 1
  for (int r = (place * kTreeJoinBlocks + blockIdx.y) * kTreeJoinWarps + warp; r < rows;
       r += (parts - 1) * kTreeJoinBlocks * kTreeJoinWarps) {
    float top = -INFINITY, sum = 0.0f, o[VL] = {};
#pragma unroll 1
    for (int p0 = 0; p0 < parts; p0 += kTreeAhead) {
      float2 ml[kTreeAhead];
      float v[kTreeAhead][VL], t = top;
#pragma unroll
      for (int i = 0; i < kTreeAhead; ++i) {
        const int p = p0 + i;
        ml[i] = make_float2(-INFINITY, 0.0f);
        if (p >= parts) break;
        const long long at = (2ll * (cta + p * size) + (p == 0 ? 0 : 1)) * ROWS + r;
        ml[i] = A.part_ml[at];
        const float* const x = A.part_o + at * DP + lane * VL;
        if constexpr (VL >= 4) {
#pragma unroll
          for (int j = 0; j < VL; j += 4)
            *reinterpret_cast<float4*>(v[i] + j) = *reinterpret_cast<const float4*>(x + j);
        } else {
          *reinterpret_cast<float2*>(v[i]) = *reinterpret_cast<const float2*>(x);
        }
      }
#pragma unroll
      for (int i = 0; i < kTreeAhead; ++i)
        if (p0 + i < parts) t = fmaxf(t, ml[i].x);
      const float g = t == -INFINITY ? 1.0f : tree_ex2(top - t);
      top = t;
      sum *= g;
#pragma unroll
      for (int j = 0; j < VL; ++j) o[j] *= g;
#pragma unroll
      for (int i = 0; i < kTreeAhead; ++i) {
        if (p0 + i >= parts) break;
        const float f = t == -INFINITY ? 1.0f : tree_ex2(ml[i].x - t);
        sum += f * ml[i].y;
#pragma unroll
        for (int j = 0; j < VL; ++j) o[j] += f * v[i][j];
      }
    }
    const float inv = top == -INFINITY ? 0.0f : mul / sum;
    const int place_in = r0 + r, node = place_in / A.group;
    const int h = kvh * A.group + place_in - node * A.group;
    const long long row = s.row0 + node, to = row * A.o_n + h * A.o_h;
#pragma unroll
    for (int j = 0; j < VL; ++j) o[j] *= inv;
    if constexpr (VL >= 4) {
#pragma unroll
      for (int j = 0; j < VL; j += 4)
        if (lane * VL + j < A.dim)
          tree_store4<KV>(A.out, to + lane * VL + j, o[j], o[j + 1], o[j + 2], o[j + 3]);
    } else {  // two lanes' columns together
      const float a = __shfl_down_sync(0xffffffffu, o[0], 1);
      const float b = __shfl_down_sync(0xffffffffu, o[1], 1);
      if (lane % 2 == 0 && lane * VL < A.dim)
        tree_store4<KV>(A.out, to + lane * VL, o[0], o[1], a, b);
    }
    if (A.lse && lane == 0) A.lse[row * A.Hq + h] = tree_lse<KV>(top, sum);
  }
}

}  // namespace moe
