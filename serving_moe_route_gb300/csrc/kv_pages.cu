// kv_pages.cu -- pages of the key-value cache that requests share, copy, move
// and give back: kv_trim, kv_fork, kv_copy_pages and kv_compact of
// include/moe_route.h.
//
// A page's word in page_refs counts the rows that hold it beyond the first, so
// that pages which nobody shares, all those of moe_kv_step, need no upkeep.
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>

#include "../../include/moe_route.h"
#include "decode_internal.cuh"
#include "moe_internal.cuh"
#include "ptx.cuh"

namespace moe {

constexpr int kPageThreads = 1024;
constexpr int kPageCtas = 8;  // a cluster that every GPU of this kind takes

// exclusive sum of one value per thread over the CTA; `total` receives the sum.
// Every thread calls it; `sums` holds 33 values.
__device__ __forceinline__ int scan1(int v, int* sums, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, off);
    if (lane >= off) x += y;
  }
  if (lane == 31) sums[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int s = sums[lane];
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, s, off);
      if (lane >= off) s += y;
    }
    sums[lane] = s;
  }
  __syncthreads();
  const int before = (warp ? sums[warp - 1] : 0) + x - v;
  total = sums[31];
  __syncthreads();
  return before;
}

__device__ __forceinline__ int pages_of(int tokens, int page, int width) {
  if (tokens <= 0) return 0;
  return min((tokens - 1) / page + 1, width);
}

// the two halves of cluster_sync
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// this CTA's value `mine` as the sum over the cluster's CTAs before it, and
// over all of them.  `inbox`: kPageCtas words of this CTA that the others write, so
// all of the cluster must have passed a barrier before
__device__ __forceinline__ int over_cluster(int mine, int* inbox, int ctas, int& total) {
  if (ctas == 1) {
    total = mine;
    return 0;
  }
  const int me = blockIdx.x;
  if (static_cast<int>(threadIdx.x) < ctas) {
    const uint32_t at = mapa_shared(smem_u32(inbox + me), threadIdx.x);
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at), "r"(mine) : "memory");
  }
  cluster_sync();
  int before = 0;
  total = 0;
  for (int c = 0; c < ctas; ++c) {
    if (c < me) before += inbox[c];
    total += inbox[c];
  }
  return before;
}

struct TrimArgs {
  const int *keep, *lens;
  int* table;
  long long table_stride;
  int* free_pages;
  int* n_free;
  int* refs;
  unsigned* err;
  int B, max_pages, free_cap, num_pages, page;
};

// The entries that rows give back, in order of rows and columns, are dealt out
// to the threads of one cluster.  With page_refs a page may be given back by
// several rows at once, and which of them frees it must not depend on who comes
// first: all take themselves off its count, and where that falls below 0 the
// first entry, by its place, marks the word as its own (minimum of INT_MIN +
// place).  Three passes over entries that a thread mostly holds; bound by latency
// and the cluster's barriers: 9.8 us for 384 rows that share up to 32 pages with
// 48 others (a cluster of eight; times in this file: caches cold).
__global__ void __launch_bounds__(kPageThreads) kv_trim_kernel(const TrimArgs A) {
  extern __shared__ int base[];  // [B] the first entry that a row gives back
  __shared__ int sums[33];
  __shared__ int inbox[kPageCtas];
  const int tid = threadIdx.x, ctas = gridDim.x;
  if (ctas > 1) cluster_arrive();  // waited for before the first write into another CTA
  pdl_wait();
  const int old = max(0, min(*A.n_free, A.free_cap));
  unsigned bad = 0;
  int entries = 0;
  for (int r0 = 0; r0 < A.B; r0 += kPageThreads) {
    const int r = r0 + tid;
    int n = 0;
    if (r < A.B)
      n = max(0, pages_of(A.lens[r], A.page, A.max_pages) -
                     pages_of(A.keep[r], A.page, A.max_pages));
    int all;
    const int before = scan1(n, sums, all);
    if (r < A.B) base[r] = entries + before;
    entries += all;
  }
  if (ctas > 1) cluster_wait();
  __syncthreads();
  // this CTA's entries
  const int share = (entries - 1) / ctas + 1;
  const int lo = min(static_cast<long long>(entries), static_cast<long long>(share) * blockIdx.x);
  const int hi = min(static_cast<long long>(entries), static_cast<long long>(lo) + share);
  auto entry = [&](int e) {
    const int r = last_at_most(base, A.B, e);
    return A.table + r * A.table_stride + pages_of(A.keep[r], A.page, A.max_pages) + (e - base[r]);
  };
  auto inside = [&](int pg) { return pg >= 0 && pg < A.num_pages; };
  // a thread's first entries are looked up once; any others in each pass
  constexpr int HOLD = 4;
  int* held[HOLD];
  int pages[HOLD];
#pragma unroll
  for (int k = 0; k < HOLD; ++k) {
    const int e = lo + k * kPageThreads + tid;
    held[k] = e < hi ? entry(e) : nullptr;
    pages[k] = e < hi ? *held[k] : -1;
  }
  auto each = [&](auto f) {  // f(entry, its page)
#pragma unroll
    for (int k = 0; k < HOLD; ++k)
      if (inside(pages[k])) f(lo + k * kPageThreads + tid, pages[k]);
    for (int e = lo + HOLD * kPageThreads + tid; e < hi; e += kPageThreads) {
      const int pg = *entry(e);
      if (inside(pg)) f(e, pg);
    }
  };
  auto all_done = [&] {
    if (ctas > 1) cluster_sync();
    else __syncthreads();
  };
  if (A.refs) {
    each([&](int, int pg) { atomicSub(A.refs + pg, 1); });
    all_done();
    each([&](int e, int pg) {
      if (__ldcg(A.refs + pg) < 0) atomicMin(A.refs + pg, INT_MIN + e);
    });
    all_done();
  }
  auto frees = [&](int e, int pg) { return !A.refs || __ldcg(A.refs + pg) == INT_MIN + e; };
  int mine = 0, mask = 0;  // of the held entries: which free their page
  each([&](int e, int pg) {
    const bool out = frees(e, pg);
    mine += out;
    const int k = (e - lo) / kPageThreads;
    if (out && k < HOLD) mask |= 1 << k;
  });
  int count, total;
  scan1(mine, sums, count);
  long long at = old + static_cast<long long>(over_cluster(count, inbox, ctas, total));
  for (int k = 0; lo + k * kPageThreads < hi; ++k) {
    const int e = lo + k * kPageThreads + tid;
    int pg = -1;
    bool out = false;
    if (e < hi) {
      int* const w = entry(e);
      pg = *w;
      out = k < HOLD ? mask >> k & 1 : inside(pg) && frees(e, pg);
      *w = -1;
      if (pg != -1 && !inside(pg)) bad |= MOE_DEVERR_BAD_PAGE;
    }
    int all;
    const long long to = at + scan1(out, sums, all);
    if (out) {
      if (to < A.free_cap) A.free_pages[to] = pg;
      if (A.refs) A.refs[pg] = 0;
    }
    at += all;
  }
  if (blockIdx.x == 0 && tid == 0) {
    const long long left = static_cast<long long>(old) + total;
    *A.n_free = static_cast<int>(min(left, static_cast<long long>(A.free_cap)));
    if (left > A.free_cap) bad |= MOE_DEVERR_NO_SPACE;
  }
  if (bad && A.err) atomicOr(A.err, bad);
}

struct ForkArgs {
  const int *src, *dst;
  int* ctx;
  int* table;
  long long table_stride;
  int* refs;
  const int* free_pages;
  int* n_free;
  int *src_pages, *dst_pages, *tokens;
  unsigned* err;
  int F, B, max_pages, free_cap, num_pages, page;
};

// Every CTA of the cluster looks all forks over (which are refused, which page
// of the free list each one's partial page is) and takes its share of the
// entries to copy.  Bound by latency: a chain of six dependent loads and a
// barrier: 8.7 us for 384 forks of up to 2048 tokens in pages of 64.
__global__ void __launch_bounds__(kPageThreads) kv_fork_kernel(const ForkArgs A) {
  extern __shared__ int fork_smem[];
  int* const claim = fork_smem;        // [B] the first fork that writes a row
  int* const base = fork_smem + A.B;   // [F] the first shared entry of a fork
  __shared__ int sums[33];
  pdl_wait();
  const int tid = threadIdx.x, ctas = gridDim.x;
  const int n_free = max(0, min(*A.n_free, A.free_cap));
  unsigned bad = 0;
  for (int r = tid; r < A.B; r += kPageThreads) claim[r] = A.F;
  __syncthreads();
  auto row = [&](int r) { return r >= 0 && r < A.B; };
  for (int i = tid; i < A.F; i += kPageThreads)
    if (row(A.dst[i])) atomicMin(claim + A.dst[i], i);
  __syncthreads();
  int shared = 0, taken = 0;
  for (int i0 = 0; i0 < A.F; i0 += kPageThreads) {
    const int i = i0 + tid;
    int s = 0, d = 0, n = 0, full = 0, part = 0;
    bool ok = false;
    if (i < A.F) {
      s = A.src[i];
      d = A.dst[i];
      if (!row(s) || !row(d)) bad |= MOE_DEVERR_BAD_ID;
      else if (claim[d] != i || claim[s] != A.F) bad |= MOE_DEVERR_DUP_ID;
      else ok = true;
      if (ok) {  // nobody writes the length of a row that is forked
        n = max(0, A.ctx[s]);
        full = n / A.page;
        part = n - full * A.page;
        if (full > A.max_pages || (full == A.max_pages && part)) {
          bad |= MOE_DEVERR_NO_SPACE;
          ok = false;
        }
      }
    }
    int from = -1, to = -1;
    if (ok && part) {  // before a free page is dealt to it, which would be lost
      from = A.table[s * A.table_stride + full];
      if (from < 0 || from >= A.num_pages) {
        bad |= MOE_DEVERR_BAD_PAGE;
        ok = false;
      }
    }
    int all;
    const int rank = taken + scan1(ok && part, sums, all);
    taken += all;
    if (ok && part) {
      if (rank < n_free) to = __ldg(A.free_pages + (n_free - 1 - rank));
      if (rank >= n_free) {
        bad |= MOE_DEVERR_NO_SPACE;
        ok = false;
      } else if (to < 0 || to >= A.num_pages) {
        bad |= MOE_DEVERR_BAD_PAGE;
        ok = false;
      }
    }
    const int before = scan1(ok ? full : 0, sums, all);
    if (i < A.F) {
      base[i] = shared + before;
      if (blockIdx.x == 0) {
        A.src_pages[i] = ok ? from : -1;
        A.dst_pages[i] = ok ? to : -1;
        A.tokens[i] = ok ? part : 0;
        if (ok) {
          if (part) A.table[d * A.table_stride + full] = to;
          A.ctx[d] = n;
        }
      }
    }
    shared += all;
  }
  __syncthreads();
  if (ctas > 1) cluster_sync();  // all have read n_free, and the lengths
  for (long long e = blockIdx.x * kPageThreads + tid; e < shared;
       e += static_cast<long long>(ctas) * kPageThreads) {
    const int i = last_at_most(base, A.F, static_cast<int>(e));
    const long long col = e - base[i];
    int pg = A.table[A.src[i] * A.table_stride + col];
    if (pg < 0 || pg >= A.num_pages) {
      bad |= MOE_DEVERR_BAD_PAGE;
      pg = -1;
    } else {
      atomicAdd(A.refs + pg, 1);
    }
    A.table[A.dst[i] * A.table_stride + col] = pg;
  }
  if (blockIdx.x == 0 && tid == 0) *A.n_free = max(0, n_free - taken);
  if (bad && A.err) atomicOr(A.err, bad);
}

// What the two kernels that move cached vectors know of the cache
struct MoveArgs {
  char* p[2];
  long long s_page, s_token, s_head;  // bytes
  const int *a, *b;                   // copy: src and dst pages; compact: path, accepted
  const int* tokens;                  // copy
  const int* ctx;                     // compact
  const int* table;
  long long table_stride;
  unsigned* err;
  int n, heads, chunks, page, num_pages;  // chunks: 16-byte pieces of a vector
  int path, max_pages;
  bool by_head;  // tokens of a head lie next to each other
};

// 16 bytes per thread and step, four steps with their loads before the first
// store.  Bound by the bytes of the copied tokens, read and written once: 384
// pages of 64 tokens, on average half filled, 4 heads of 128, bf16: 11.6 us, 4.3
// TB/s.
constexpr int kMoveThreads = 256;
constexpr int kMoveSteps = 4;
__global__ void __launch_bounds__(kMoveThreads) kv_copy_pages_kernel(const MoveArgs A) {
  pdl_wait();
  const unsigned per_token = static_cast<unsigned>(A.heads) * A.chunks;
  for (int i = blockIdx.y; i < A.n; i += gridDim.y) {
    const int from = A.a[i], to = A.b[i];
    if (from == -1 || to == -1) continue;
    if (from < 0 || from >= A.num_pages || to < 0 || to >= A.num_pages) {
      if (A.err && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(A.err, MOE_DEVERR_BAD_PAGE);
      continue;
    }
    if (from == to) continue;
    const int tokens = A.tokens ? max(0, min(A.tokens[i], A.page)) : A.page;
    const long long half = static_cast<long long>(tokens) * per_token, total = 2 * half;
    const long long step = static_cast<long long>(gridDim.x) * kMoveThreads;
    for (long long x0 = static_cast<long long>(blockIdx.x) * kMoveThreads + threadIdx.x; x0 < total;
         x0 += step * kMoveSteps) {
      uint4 v[kMoveSteps];
      char* out[kMoveSteps];
#pragma unroll
      for (int u = 0; u < kMoveSteps; ++u) {
        const long long x = x0 + u * step;
        out[u] = nullptr;
        if (x >= total) continue;
        const int which = x >= half;
        const long long y = x - which * half;
        long long outer, c;
        if (half <= UINT_MAX) {
          outer = static_cast<unsigned>(y) / A.chunks;
          c = y - outer * A.chunks;
        } else {
          outer = y / A.chunks;
          c = y - outer * A.chunks;
        }
        long long h, t;
        if (A.by_head) {
          h = outer / tokens;
          t = outer - h * tokens;
        } else {
          t = outer / A.heads;
          h = outer - t * A.heads;
        }
        const long long off = t * A.s_token + h * A.s_head + c * 16;
        out[u] = A.p[which] + to * A.s_page + off;
        v[u] = *reinterpret_cast<const uint4*>(A.p[which] + from * A.s_page + off);
      }
#pragma unroll
      for (int u = 0; u < kMoveSteps; ++u)
        if (out[u]) *reinterpret_cast<uint4*>(out[u]) = v[u];
    }
  }
}

// A thread owns one 16-byte column (of keys or values, of a head) of a request
// and moves its accepted tokens in order.  Token j goes to place j <= path[j], and
// the path rises, so no move overwrites what a later one reads: no staging, no
// barrier between moves.  Bound by latency (lengths, path, pages, values): 8.6 us
// for 128 requests of 64 nodes.
constexpr int kPathThreads = 128;
constexpr int kPathSteps = 4;
__global__ void __launch_bounds__(kPathThreads) kv_compact_kernel(const MoveArgs A) {
  __shared__ long long s_from[kPathThreads], s_to[kPathThreads];
  __shared__ int s_stop;
  pdl_wait();
  const int tid = threadIdx.x;
  const int r = blockIdx.x;
  const int count = max(0, min(A.b[r], A.path));
  const int ctx = max(0, A.ctx[r]);
  const int* const path = A.a + static_cast<long long>(r) * A.path;
  const int columns = 2 * A.heads * A.chunks;
  unsigned bad = 0;
  for (int j0 = 0; j0 < count; j0 += kPathThreads) {
    if (tid == 0) s_stop = min(kPathThreads, count - j0);
    __syncthreads();
    const int j = j0 + tid;
    long long from = -1, to = -1;
    if (j < count) {
      const int p = path[j];
      if (p < j || (j > 0 && path[j - 1] >= p)) {  // not a rising path: it ends here
        bad |= MOE_DEVERR_BAD_ID;
        atomicMin(&s_stop, tid);
      } else if (p != j) {
        auto place = [&](long long pos) -> long long {
          const long long col = pos / A.page;
          if (col >= A.max_pages) {
            bad |= MOE_DEVERR_NO_SPACE;
            return -1;
          }
          const int pg = A.table[r * A.table_stride + col];
          if (pg < 0 || pg >= A.num_pages) {
            bad |= MOE_DEVERR_BAD_PAGE;
            return -1;
          }
          return pg * A.s_page + (pos - col * A.page) * A.s_token;
        };
        from = place(static_cast<long long>(ctx) + p);
        to = place(static_cast<long long>(ctx) + j);
        if (to < 0) from = -1;
      }
    }
    s_from[tid] = from;
    s_to[tid] = to;
    __syncthreads();
    const int stop = s_stop;
    for (int x = blockIdx.y * kPathThreads + tid; x < columns; x += gridDim.y * kPathThreads) {
      const int which = x >= columns / 2;
      const int y = x - which * (columns / 2);
      const int h = y / A.chunks, c = y - h * A.chunks;
      char* const column = A.p[which] + h * A.s_head + c * 16;
      for (int k = 0; k < stop; k += kPathSteps) {
        uint4 v[kPathSteps];
#pragma unroll
        for (int u = 0; u < kPathSteps; ++u)
          if (k + u < stop && s_from[k + u] >= 0)
            v[u] = *reinterpret_cast<const uint4*>(column + s_from[k + u]);
#pragma unroll
        for (int u = 0; u < kPathSteps; ++u)
          if (k + u < stop && s_from[k + u] >= 0)
            *reinterpret_cast<uint4*>(column + s_to[k + u]) = v[u];
      }
    }
    if (stop < min(kPathThreads, count - j0)) break;
    __syncthreads();
  }
  if (bad && A.err && blockIdx.y == 0) atomicOr(A.err, bad);
}

// MOE_OK if the cache's vectors may be moved: no two of them share memory.  Their
// bytes stay what they are, so the scales need not be there
static int movable(const moe_kv_cache_t* c) {
  if (!c) return MOE_ERR_INVALID_ARG;
  moe_kv_cache_t any = *c;
  static const float one = 1.0f;
  any.k_scale = any.v_scale = c->kv_dtype == MOE_KV_E4M3 ? &one : nullptr;
  const int rc = kv_cache_ok(&any);
  if (rc != MOE_OK) return rc;
  if (c->k == c->v || !apart(c->num_pages, c->stride_page, c->head_dim) ||
      !apart(c->page_size, c->stride_token, c->head_dim) ||
      !apart(c->kv_heads, c->stride_head, c->head_dim))
    return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

static MoveArgs move_args(const moe_kv_cache_t* c) {
  const int es = kv_esize(c->kv_dtype);
  MoveArgs a = {};
  a.p[0] = static_cast<char*>(c->k);
  a.p[1] = static_cast<char*>(c->v);
  a.s_page = c->stride_page * es;
  a.s_token = c->stride_token * es;
  a.s_head = c->stride_head * es;
  a.heads = c->kv_heads;
  a.chunks = c->head_dim * es / 16;
  a.page = c->page_size;
  a.num_pages = c->num_pages;
  a.by_head = c->kv_heads > 1 && c->stride_head > c->stride_token;
  return a;
}

static bool table_ok(int B, int max_pages, long long table_stride) {
  return B >= 0 && B <= MOE_KV_MAX_REQUESTS && max_pages >= 1 && table_stride >= max_pages;
}

}  // namespace moe

using namespace moe;

extern "C" {

int moe_kv_trim(const int32_t* keep_lens, const int32_t* seq_lens, int B, int32_t* block_table,
                int max_pages, long long table_stride, int32_t* free_pages, int free_capacity,
                int32_t* n_free, int32_t* page_refs, int num_pages, int page_size, uint32_t* err,
                void* stream) {
  if (!table_ok(B, max_pages, table_stride) || free_capacity < 0 || num_pages < 1 || page_size < 1 ||
      static_cast<long long>(num_pages) * page_size > INT_MAX ||
      static_cast<long long>(B) * max_pages >= INT_MAX - 8 * kPageThreads)
    return MOE_ERR_INVALID_ARG;
  if (B == 0) return MOE_OK;
  if (!keep_lens || !seq_lens || !block_table || !n_free || (free_capacity > 0 && !free_pages))
    return MOE_ERR_INVALID_ARG;
  const TrimArgs a = {keep_lens, seq_lens, block_table, table_stride, free_pages, n_free, page_refs,
                      err, B, max_pages, free_capacity, num_pages, page_size};
  const int ctas = static_cast<long long>(B) * max_pages > kPageThreads ? kPageCtas : 1;
  return launch_cluster(kv_trim_kernel, dim3(ctas), dim3(kPageThreads), ctas,
                        static_cast<size_t>(B) * sizeof(int), static_cast<cudaStream_t>(stream),
                        a) == cudaSuccess
             ? MOE_OK
             : MOE_ERR_CUDA;
}

int moe_kv_fork(const int32_t* src_rows, const int32_t* dst_rows, int F, int32_t* ctx_lens, int B,
                int32_t* block_table, int max_pages, long long table_stride, int32_t* page_refs,
                const int32_t* free_pages, int free_capacity, int32_t* n_free, int num_pages,
                int page_size, int32_t* src_pages, int32_t* dst_pages, int32_t* tokens,
                uint32_t* err, void* stream) {
  if (!table_ok(B, max_pages, table_stride) || F < 0 || F > MOE_KV_MAX_REQUESTS ||
      free_capacity < 0 || num_pages < 1 || page_size < 1 ||
      static_cast<long long>(num_pages) * page_size > INT_MAX ||
      static_cast<long long>(F) * max_pages >= INT_MAX)
    return MOE_ERR_INVALID_ARG;
  if (F == 0) return MOE_OK;
  if (B == 0 || !src_rows || !dst_rows || !ctx_lens || !block_table || !page_refs || !n_free ||
      !src_pages || !dst_pages || !tokens || (free_capacity > 0 && !free_pages))
    return MOE_ERR_INVALID_ARG;
  const ForkArgs a = {src_rows, dst_rows, ctx_lens, block_table, table_stride, page_refs, free_pages,
                      n_free, src_pages, dst_pages, tokens, err, F, B, max_pages, free_capacity,
                      num_pages, page_size};
  const size_t smem = (static_cast<size_t>(B) + F) * sizeof(int);
  static std::atomic<uint64_t> done{0};
  if (smem > 32 * 1024 &&
      allow_smem(reinterpret_cast<const void*>(kv_fork_kernel),
                 2 * MOE_KV_MAX_REQUESTS * static_cast<int>(sizeof(int)), done) != cudaSuccess)
    return MOE_ERR_CUDA;
  const int ctas = static_cast<long long>(F) * max_pages > kPageThreads ? kPageCtas : 1;
  return launch_cluster(kv_fork_kernel, dim3(ctas), dim3(kPageThreads), ctas, smem,
                        static_cast<cudaStream_t>(stream), a) == cudaSuccess
             ? MOE_OK
             : MOE_ERR_CUDA;
}

int moe_kv_copy_pages(const moe_kv_cache_t* cache, const int32_t* src_pages,
                      const int32_t* dst_pages, const int32_t* tokens, int n, uint32_t* err,
                      void* stream) {
  const int rc = movable(cache);
  if (rc != MOE_OK) return rc;
  if (n < 0) return MOE_ERR_INVALID_ARG;
  if (n == 0) return MOE_OK;
  if (!src_pages || !dst_pages) return MOE_ERR_INVALID_ARG;
  MoveArgs a = move_args(cache);
  a.a = src_pages;
  a.b = dst_pages;
  a.tokens = tokens;
  a.err = err;
  a.n = n;
  // a page's pieces over enough CTAs that each thread has about four
  const long long pieces = 2ll * a.page * a.heads * a.chunks;
  const long long want = (pieces + kMoveThreads * kMoveSteps - 1) / (kMoveThreads * kMoveSteps);
  const dim3 grid(static_cast<unsigned>(want < 1024 ? want : 1024), n < 65535 ? n : 65535);
  return launch_chained(kv_copy_pages_kernel, grid, dim3(kMoveThreads), 0,
                        static_cast<cudaStream_t>(stream), a) == cudaSuccess
             ? MOE_OK
             : MOE_ERR_CUDA;
}

int moe_kv_compact(const moe_kv_cache_t* cache, const int32_t* path, int max_path,
                   const int32_t* accepted, const int32_t* ctx_lens, int B,
                   const int32_t* block_table, int max_pages, long long table_stride,
                   uint32_t* err, void* stream) {
  const int rc = movable(cache);
  if (rc != MOE_OK) return rc;
  if (!table_ok(B, max_pages, table_stride) || max_path < 1 || max_path > INT_MAX - kPathThreads)
    return MOE_ERR_INVALID_ARG;
  if (B == 0) return MOE_OK;
  if (!path || !accepted || !ctx_lens || !block_table) return MOE_ERR_INVALID_ARG;
  MoveArgs a = move_args(cache);
  a.a = path;
  a.b = accepted;
  a.path = max_path;
  a.ctx = ctx_lens;
  a.table = block_table;
  a.table_stride = table_stride;
  a.max_pages = max_pages;
  a.err = err;
  const long long columns = 2ll * a.heads * a.chunks;
  const long long want = (columns + kPathThreads - 1) / kPathThreads;
  return launch_chained(kv_compact_kernel, dim3(B, want < 1024 ? want : 1024), dim3(kPathThreads),
                        0, static_cast<cudaStream_t>(stream), a) == cudaSuccess
             ? MOE_OK
             : MOE_ERR_CUDA;
}

}  // extern "C"
