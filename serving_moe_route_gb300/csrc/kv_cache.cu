// kv_cache.cu -- the paged key-value cache around the layer: block tables and
// slot maps from request lengths (moe_kv_step), the return of finished
// requests' pages (moe_kv_release) and the write of new keys and values
// (moe_kv_append).  The layout is described in include/moe_route.h.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>

#include "../../include/moe_route.h"
#include "decode_internal.cuh"
#include "moe_internal.cuh"
#include "ptx.cuh"

namespace moe {

constexpr int kStepThreads = 1024;

// exclusive sums of two values per thread over the CTA; tot_a / tot_b
// receive the sums.  Every thread calls it.
__device__ void scan2(long long a, long long b, long long* sums, long long& ex_a, long long& ex_b,
                      long long& tot_a, long long& tot_b) {
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
    sums[32 + warp] = y;
  }
  __syncthreads();
  if (warp < 2) {
    const int nw = blockDim.x >> 5;
    long long s = lane < nw ? sums[32 * warp + lane] : 0;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, s, off);
      if (lane >= off) s += u;
    }
    sums[32 * warp + lane] = s;
  }
  __syncthreads();
  ex_a = (warp ? sums[warp - 1] : 0) + x - a;
  ex_b = (warp ? sums[32 + warp - 1] : 0) + y - b;
  tot_a = sums[31];
  tot_b = sums[63];
  __syncthreads();
}

struct StepArgs {
  const int* ctx;
  const int* nw;
  int* table;
  const int* free_pages;
  const int* n_free_in;
  int* n_free_out;
  int *slots, *positions, *starts, *seq_lens;
  unsigned* err;
  long long table_stride;
  int B, max_pages, free_cap, num_pages, page, page_shift, max_tokens;
};

__device__ __forceinline__ int cut_int(long long v) {
  return v > INT_MAX ? INT_MAX : static_cast<int>(v);
}

// Every CTA scans the requests' new tokens and new pages for itself (two
// exclusive sums, at most 8 steps of 1024 requests) and keeps them in shared
// memory; then the token rows and the new table entries are dealt out over
// all threads, each of which finds its request by bisection.  A new page's id
// is taken straight from the free list by its rank, so no thread waits for
// another's table entry.  Bound by latency (a few dependent loads).  If
// n_free_out is n_free_in, the CTAs are one cluster and all read it before one
// writes it; else there may be any number of them.
__global__ void __launch_bounds__(kStepThreads) kv_step_kernel(const StepArgs A, bool cluster) {
  extern __shared__ int step_smem[];
  int* const start = step_smem;           // [B] first token row
  int* const base = step_smem + A.B;      // [B] rank of the first new page
  int* const ctx = step_smem + 2 * A.B;   // [B]
  __shared__ long long sums[64];
  pdl_wait();
  const int tid = threadIdx.x, cta = blockIdx.x, nthreads = kStepThreads * gridDim.x;
  const int n_free = max(0, min(*A.n_free_in, A.free_cap));
  const int W = A.max_pages;
  const unsigned P = A.page;
  // below 2^32: a context and its new tokens both fit an int
  auto page_of = [&](unsigned pos) { return A.page_shift >= 0 ? pos >> A.page_shift : pos / P; };
  auto pages_for = [&](unsigned n) {
    return n ? min(page_of(n - 1) + 1u, static_cast<unsigned>(W)) : 0u;
  };
  unsigned bad = 0;
  long long tokens = 0, pages = 0;
  for (int r0 = 0; r0 < A.B; r0 += kStepThreads) {
    const int r = r0 + tid;
    int c = 0, n = 0, take = 0;
    if (r < A.B) {
      c = max(A.ctx[r], 0);
      n = max(A.nw[r], 0);
      const unsigned all = static_cast<unsigned>(c) + static_cast<unsigned>(n);
      take = static_cast<int>(pages_for(all) - pages_for(c));
      if (n > 0 && page_of(all - 1) >= static_cast<unsigned>(W)) bad |= MOE_DEVERR_NO_SPACE;
    }
    long long ex_t, ex_p, tot_t, tot_p;
    scan2(n, take, sums, ex_t, ex_p, tot_t, tot_p);
    if (r < A.B) {
      start[r] = cut_int(tokens + ex_t);
      base[r] = cut_int(pages + ex_p);
      ctx[r] = c;
      if (cta == 0) {
        A.starts[r] = start[r];
        A.seq_lens[r] = cut_int(static_cast<long long>(c) + n);
      }
    }
    tokens += tot_t;
    pages += tot_p;
  }
  __syncthreads();
  if (cluster) cluster_sync();
  if (cta == 0 && tid == 0) {
    A.starts[A.B] = cut_int(tokens);
    *A.n_free_out = static_cast<int>(max(0ll, n_free - pages));
    if (tokens > A.max_tokens || pages > n_free) bad |= MOE_DEVERR_NO_SPACE;
  }
  // the page of rank `rank` among the new ones, -1 where there is none
  auto fresh = [&](long long rank) {
    if (rank >= n_free) return -1;
    const int id = __ldg(A.free_pages + (n_free - 1 - rank));
    if (id >= 0 && id < A.num_pages) return id;
    bad |= MOE_DEVERR_BAD_PAGE;
    return -1;
  };
  for (int i = cta * kStepThreads + tid; i < A.max_tokens; i += nthreads) {
    int slot = -1, pos = 0;
    if (i < tokens) {
      const int r = last_at_most(start, A.B, i);
      const unsigned c = ctx[r], p = c + static_cast<unsigned>(i - start[r]), col = page_of(p);
      pos = cut_int(p);
      if (col < static_cast<unsigned>(W)) {
        const unsigned have = pages_for(c);
        int id;
        if (col < have) {
          id = A.table[r * A.table_stride + col];
          if (id < 0 || id >= A.num_pages) {
            id = -1;
            bad |= MOE_DEVERR_BAD_PAGE;
          }
        } else {
          id = fresh(static_cast<long long>(base[r]) + col - have);
        }
        if (id >= 0) slot = id * static_cast<int>(P) + static_cast<int>(p - col * P);
      }
    }
    A.slots[i] = slot;
    A.positions[i] = pos;
    if (i > INT_MAX - nthreads) break;
  }
  // ranks from 2^31 - 1 on are no ints: there is no page for them, and no entry
  // of theirs is touched
  const long long ranks = min(pages, static_cast<long long>(INT_MAX));
  for (long long i = static_cast<long long>(cta) * kStepThreads + tid; i < ranks; i += nthreads) {
    const int r = last_at_most(base, A.B, cut_int(i));
    const long long col = static_cast<long long>(pages_for(ctx[r])) + i - base[r];
    A.table[r * A.table_stride + col] = fresh(i);
  }
  if (bad && A.err) atomicOr(A.err, bad);
}

// One CTA: a warp counts the pages of a finished row, a scan over the rows
// places them, and the warps copy them to the end of the list.  Bound by the
// latency of a row's columns, 32 at a time, count and copy: 4.5 us for 8 of 256
// requests with 64 columns, 10 for 64 of 256 with 512, 60 for one of 16384.
__global__ void __launch_bounds__(1024)
    kv_release_kernel(const int* __restrict__ done, int B, int* __restrict__ table, int max_pages,
                      long long table_stride, int* __restrict__ free_pages, int free_cap,
                      int* __restrict__ n_free, int num_pages, unsigned* err) {
  extern __shared__ int count[];  // [B] pages of a finished row, then its place
  __shared__ long long sums[64];
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int old = max(0, min(*n_free, free_cap));
  for (int r = warp; r < B; r += 32) {
    int n = 0;
    if (done[r]) {
      const int* row = table + r * table_stride;
      for (int c = lane; c < max_pages; c += 32) n += row[c] >= 0 && row[c] < num_pages;
      n = __reduce_add_sync(0xffffffffu, n);
    }
    if (lane == 0) count[r] = n;
  }
  __syncthreads();
  long long at = old;
  for (int r0 = 0; r0 < B; r0 += 1024) {
    const int r = r0 + threadIdx.x;
    const int n = r < B ? count[r] : 0;
    long long ex, unused, tot, tot_b;
    scan2(n, 0, sums, ex, unused, tot, tot_b);
    if (r < B) count[r] = cut_int(at + ex);
    at += tot;
  }
  __syncthreads();
  for (int r = warp; r < B; r += 32) {
    if (!done[r]) continue;
    int* row = table + r * table_stride;
    long long to = count[r];
    for (int c0 = 0; c0 < max_pages; c0 += 32) {
      const int c = c0 + lane;
      const int id = c < max_pages ? row[c] : -1;
      const bool ok = id >= 0 && id < num_pages;
      const unsigned m = __ballot_sync(0xffffffffu, ok);
      const long long mine = to + __popc(m & ((1u << lane) - 1));
      if (ok && mine < free_cap) free_pages[mine] = id;
      if (c < max_pages) row[c] = -1;
      to += __popc(m);
    }
  }
  if (threadIdx.x == 0) {
    *n_free = static_cast<int>(min(at, static_cast<long long>(free_cap)));
    if (at > free_cap && err) atomicOr(err, MOE_DEVERR_NO_SPACE);
  }
}

struct AppendArgs {
  const char* src[2];
  long long src_t[2], src_h[2];  // bytes
  char* dst[2];
  const float* scale[2];
  long long dst_page, dst_t, dst_h;  // bytes
  const int* slots;
  unsigned* err;
  int N, heads, dim, page, num_pages;
  bool vec;  // source rows are 16-byte aligned
};

// 16 bytes of cached vectors per thread and step (blockIdx.y: keys, values), U
// steps with all their loads before the first store; bound by its bytes: a
// source vector is read once and a cached one written once.  16384 tokens of 8
// heads of 128, bf16, to scattered slots: 26.3 us, 5.1 TB/s.
constexpr int kAppendThreads = 256;
template <int KV, int U>
__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(const AppendArgs A) {
  constexpr int ES = kv_esize(KV), QS = KV == MOE_KV_F32 ? 4 : 2;
  constexpr int VE = 16 / ES;            // elements per thread
  constexpr int LD = VE * QS / 16;       // 16-byte source loads
  pdl_wait();
  const int which = blockIdx.y;
  const unsigned per_head = A.dim / VE;
  const unsigned per_token = static_cast<unsigned>(A.heads) * per_head;
  const long long total = static_cast<long long>(A.N) * per_token;
  const long long i0 = static_cast<long long>(blockIdx.x) * kAppendThreads * U + threadIdx.x;
  unsigned h[U], c[U];
  int slot[U];
  uint4 raw[U][LD];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const long long i = i0 + u * kAppendThreads;
    slot[u] = -1;
    if (i < total) {
      // 32-bit division where it does
      const long long t = total <= UINT_MAX ? static_cast<unsigned>(i) / per_token : i / per_token;
      const unsigned in = static_cast<unsigned>(i - t * per_token);
      h[u] = in / per_head;
      c[u] = in - h[u] * per_head;
      slot[u] = __ldg(A.slots + t);
      const char* s = A.src[which] + t * A.src_t[which] + h[u] * A.src_h[which] +
                      static_cast<size_t>(c[u]) * VE * QS;
      if (A.vec) {
#pragma unroll
        for (int j = 0; j < LD; ++j) raw[u][j] = __ldg(reinterpret_cast<const uint4*>(s) + j);
      } else {
        using ET = typename std::conditional<QS == 4, uint32_t, uint16_t>::type;
        ET* e = reinterpret_cast<ET*>(raw[u]);
#pragma unroll
        for (int j = 0; j < VE; ++j) e[j] = __ldg(reinterpret_cast<const ET*>(s) + j);
      }
      if (slot[u] != -1 && (slot[u] < 0 || slot[u] / A.page >= A.num_pages)) {
        slot[u] = -1;
        if (A.err && in == 0) atomicOr(A.err, MOE_DEVERR_BAD_PAGE);
      }
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (slot[u] < 0) continue;
    const int pg = slot[u] / A.page;
    uint4 out;
    if constexpr (KV == MOE_KV_E4M3) {
      const float sc = __ldg(A.scale[which] + h[u]);
      const uint32_t* w = reinterpret_cast<const uint32_t*>(raw[u]);
      __nv_fp8x2_storage_t q[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float2 v;
        v.x = __uint_as_float(w[j] << 16) / sc;
        v.y = __uint_as_float(w[j] & 0xffff0000u) / sc;
        q[j] = __nv_cvt_float2_to_fp8x2(v, __NV_SATFINITE, __NV_E4M3);
      }
      out = *reinterpret_cast<const uint4*>(q);
    } else {
      out = raw[u][0];
    }
    char* d = A.dst[which] + pg * A.dst_page + (slot[u] - pg * A.page) * A.dst_t +
              h[u] * A.dst_h + static_cast<size_t>(c[u]) * 16;
    *reinterpret_cast<uint4*>(d) = out;
  }
}

template <int KV>
static cudaError_t launch_append(const AppendArgs& a, long long items, cudaStream_t st) {
  // One step a thread, or four where there are 32 CTAs of one for each SM and
  // no conversion between load and store.  Tokens of 8 heads of 128, us:
  //            bf16, 4096   16384   f32, 4096   16384   e4m3, 4096   16384
  //   one             7.7    26.5        14.7    53.1          7.4    25.6
  //   four            8.6    26.3        14.8    50.2          9.3    30.1
  constexpr int U = 4;
  const long long one = (items + kAppendThreads - 1) / kAppendThreads;
  if constexpr (KV != MOE_KV_E4M3)
    if (one >= 32ll * sm_count())
      return launch_chained(kv_append_kernel<KV, U>,
                            dim3(static_cast<unsigned>((one + U - 1) / U), 2), dim3(kAppendThreads),
                            0, st, a);
  return launch_chained(kv_append_kernel<KV, 1>, dim3(static_cast<unsigned>(one), 2),
                        dim3(kAppendThreads), 0, st, a);
}

int kv_cache_ok(const moe_kv_cache_t* c) {
  if (!c || !c->k || !c->v) return MOE_ERR_INVALID_ARG;
  if (c->kv_dtype < MOE_KV_F32 || c->kv_dtype > MOE_KV_E4M3) return MOE_ERR_INVALID_ARG;
  if (c->num_pages < 1 || c->page_size < 1 || c->kv_heads < 1 || c->kv_heads > 65535 ||
      static_cast<long long>(c->num_pages) * c->page_size > INT_MAX)
    return MOE_ERR_INVALID_ARG;
  const bool q8 = c->kv_dtype == MOE_KV_E4M3;
  if (q8 ? (!c->k_scale || !c->v_scale) : (c->k_scale || c->v_scale)) return MOE_ERR_INVALID_ARG;
  if (c->head_dim < 1 || c->stride_page < 0 || c->stride_token < 0 || c->stride_head < 0)
    return MOE_ERR_INVALID_ARG;
  const int es = kv_esize(c->kv_dtype);
  if (c->head_dim > 256 || c->head_dim % kv_dim_step(c->kv_dtype)) return MOE_ERR_UNSUPPORTED;
  if ((c->stride_page * es) % 16 || (c->stride_token * es) % 16 || (c->stride_head * es) % 16 ||
      (reinterpret_cast<uintptr_t>(c->k) & 15) || (reinterpret_cast<uintptr_t>(c->v) & 15))
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

}  // namespace moe

using namespace moe;

extern "C" {

int moe_kv_step(const int32_t* ctx_lens, const int32_t* new_lens, int B, int32_t* block_table,
                int max_pages, long long table_stride, const int32_t* free_pages,
                int free_capacity, const int32_t* n_free_in, int32_t* n_free_out, int num_pages,
                int page_size, int max_tokens, int32_t* slots, int32_t* positions,
                int32_t* starts, int32_t* seq_lens, uint32_t* err, void* stream) {
  if (B < 0 || B > MOE_KV_MAX_REQUESTS || max_pages < 1 || table_stride < max_pages ||
      free_capacity < 0 || num_pages < 1 || page_size < 1 || max_tokens < 0 ||
      static_cast<long long>(num_pages) * page_size > INT_MAX)
    return MOE_ERR_INVALID_ARG;
  if (!n_free_in || !n_free_out || !starts) return MOE_ERR_INVALID_ARG;
  if (B > 0 && (!ctx_lens || !new_lens || !block_table || !seq_lens)) return MOE_ERR_INVALID_ARG;
  if (max_tokens > 0 && (!slots || !positions)) return MOE_ERR_INVALID_ARG;
  if (free_capacity > 0 && !free_pages) return MOE_ERR_INVALID_ARG;
  int shift = -1;
  for (int i = 0; i < 31; ++i)
    if (page_size == 1 << i) shift = i;
  const StepArgs a = {ctx_lens, new_lens, block_table, free_pages, n_free_in, n_free_out, slots,
                      positions, starts, seq_lens, err, table_stride, B, max_pages, free_capacity,
                      num_pages, page_size, shift, max_tokens};
  // a token row a thread, up to the eight CTAs that every GPU of this kind
  // takes as a cluster, or 64 where none is needed (32768 rows: 4.1 us with 32
  // CTAs)
  const bool in_place = n_free_in == n_free_out;
  const long long want = (static_cast<long long>(max_tokens) + kStepThreads - 1) / kStepThreads;
  int ctas = 1;
  if (in_place)
    while (ctas < 8 && want > ctas) ctas *= 2;
  else
    ctas = static_cast<int>(want < 1 ? 1 : want < 64 ? want : 64);
  const size_t smem = static_cast<size_t>(B) * 3 * sizeof(int);
  static std::atomic<uint64_t> done{0};
  if (smem > 32 * 1024 &&
      allow_smem(reinterpret_cast<const void*>(kv_step_kernel),
                 MOE_KV_MAX_REQUESTS * 3 * static_cast<int>(sizeof(int)), done) != cudaSuccess)
    return MOE_ERR_CUDA;
  const bool cluster = in_place && ctas > 1;
  return launch_cluster(kv_step_kernel, dim3(ctas), dim3(kStepThreads), cluster ? ctas : 1, smem,
                        static_cast<cudaStream_t>(stream), a, cluster) == cudaSuccess
             ? MOE_OK
             : MOE_ERR_CUDA;
}

int moe_kv_release(const int32_t* done, int B, int32_t* block_table, int max_pages,
                   long long table_stride, int32_t* free_pages, int free_capacity,
                   int32_t* n_free, int num_pages, uint32_t* err, void* stream) {
  if (B < 0 || B > MOE_KV_MAX_REQUESTS || max_pages < 1 || table_stride < max_pages ||
      free_capacity < 0 || num_pages < 1)
    return MOE_ERR_INVALID_ARG;
  if (B == 0) return MOE_OK;
  if (!done || !block_table || !n_free || (free_capacity > 0 && !free_pages))
    return MOE_ERR_INVALID_ARG;
  return launch_chained(kv_release_kernel, dim3(1), dim3(1024), static_cast<size_t>(B) * sizeof(int),
                        static_cast<cudaStream_t>(stream), done, B, block_table, max_pages,
                        table_stride, free_pages, free_capacity, n_free, num_pages,
                        err) == cudaSuccess
             ? MOE_OK
             : MOE_ERR_CUDA;
}

int moe_kv_append(const moe_kv_cache_t* cache, const void* k, long long k_stride_token,
                  long long k_stride_head, const void* v, long long v_stride_token,
                  long long v_stride_head, int N, const int32_t* slots, uint32_t* err,
                  void* stream) {
  const int rc = kv_cache_ok(cache);
  if (rc != MOE_OK) return rc;
  if (N < 0 || k_stride_token < 0 || k_stride_head < 0 || v_stride_token < 0 || v_stride_head < 0)
    return MOE_ERR_INVALID_ARG;
  if (N == 0) return MOE_OK;
  if (!k || !v || !slots) return MOE_ERR_INVALID_ARG;
  // what is written must not overlap: two writers of one place race
  if (cache->k == cache->v || !apart(cache->num_pages, cache->stride_page, cache->head_dim) ||
      !apart(cache->page_size, cache->stride_token, cache->head_dim) ||
      !apart(cache->kv_heads, cache->stride_head, cache->head_dim))
    return MOE_ERR_INVALID_ARG;
  const int es = kv_esize(cache->kv_dtype), qs = cache->kv_dtype == MOE_KV_F32 ? 4 : 2;
  if ((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) & (qs - 1))
    return MOE_ERR_INVALID_ARG;
  AppendArgs a = {};
  a.src[0] = static_cast<const char*>(k);
  a.src[1] = static_cast<const char*>(v);
  a.src_t[0] = k_stride_token * qs;
  a.src_h[0] = k_stride_head * qs;
  a.src_t[1] = v_stride_token * qs;
  a.src_h[1] = v_stride_head * qs;
  a.vec = ((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v) |
            static_cast<uintptr_t>(a.src_t[0] | a.src_h[0] | a.src_t[1] | a.src_h[1])) &
           15) == 0;
  a.dst[0] = static_cast<char*>(cache->k);
  a.dst[1] = static_cast<char*>(cache->v);
  a.scale[0] = cache->k_scale;
  a.scale[1] = cache->v_scale;
  a.dst_page = cache->stride_page * es;
  a.dst_t = cache->stride_token * es;
  a.dst_h = cache->stride_head * es;
  a.slots = slots;
  a.err = err;
  a.N = N;
  a.heads = cache->kv_heads;
  a.dim = cache->head_dim;
  a.page = cache->page_size;
  a.num_pages = cache->num_pages;
  const long long items = static_cast<long long>(N) * a.heads * (a.dim * es / 16);
  if (items / kAppendThreads >= INT_MAX) return MOE_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = cache->kv_dtype == MOE_KV_F32    ? launch_append<MOE_KV_F32>(a, items, st)
                        : cache->kv_dtype == MOE_KV_BF16 ? launch_append<MOE_KV_BF16>(a, items, st)
                                                         : launch_append<MOE_KV_E4M3>(a, items, st);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

int moe_check_word(uint32_t* err, uint32_t* bits, void* stream) {
  if (!err) return MOE_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint32_t word = 0;
  if (cudaMemcpyAsync(&word, err, sizeof(word), cudaMemcpyDeviceToHost, st) != cudaSuccess)
    return MOE_ERR_CUDA;
  if (cudaStreamSynchronize(st) != cudaSuccess) return MOE_ERR_CUDA;
  if (word && cudaMemsetAsync(err, 0, sizeof(uint32_t), st) != cudaSuccess) return MOE_ERR_CUDA;
  if (bits) *bits = word;
  return word ? MOE_ERR_DEVICE : MOE_OK;
}

}  // extern "C"
