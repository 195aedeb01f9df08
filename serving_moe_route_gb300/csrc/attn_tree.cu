// attn_tree.cu -- attention of several drafted tokens per request over the paged
// cache (moe_attn_tree, include/moe_route.h): the host's side, and the kernel for
// f32 caches; bf16 and e4m3 caches go to attn_tree_tc.cu.
#include "attn_tree.cuh"
#include "attn_tree_tc.cuh"

namespace moe {

constexpr int kSimtRows = 32;
constexpr int kSimtThreads = 256;
constexpr int kSimtEnd = 1;
template <int DP>
struct SimtCfg {
  static constexpr int TILE = DP == 256 ? 32 : 64;
  static constexpr int KP = DP + 4, PP = TILE + 4;  // pitches without bank conflicts
  static constexpr int SMEM = 4 * (kSimtRows * KP + TILE * KP + TILE * DP + kSimtRows * PP);
  static constexpr int CTAS = 2;  // per SM
};

// S = Q K^T, the running softmax and O += P V on tiles in shared memory, 2 rows
// by TILE / 16 tokens and by DP / 16 columns a thread, all in fp32: nothing is
// split or rounded.  A value that a row does not attend is skipped, not
// multiplied by 0.  (Tensor cores would take f32 operands as pairs of tf32 terms,
// three products each, and split them again for every block of rows.)  Bound by
// latency for small calls, 25 us for 5 requests of up to 13 nodes, 3 heads on
// each of 2 of 80, window 1000; by the fp32 units for large ones, 839 us for 64 of up
// to 16 nodes, 8 heads on each of 4 of 128, up to 4096 tokens.
template <int DP>
__global__ void __launch_bounds__(kSimtThreads, SimtCfg<DP>::CTAS)
    tree_simt_kernel(const TreeArgs A) {
  using C = SimtCfg<DP>;
  constexpr int TILE = C::TILE, KP = C::KP, PP = C::PP, NK = TILE / 16, NC = DP / 64;
  extern __shared__ __align__(16) float simt_smem[];
  float* const qs = simt_smem;
  float* const ks = qs + kSimtRows * KP;
  float* const vs = ks + TILE * KP;
  float* const ps = vs + TILE * DP;
  __shared__ TreeStart start;
  __shared__ long long sums[33];
  __shared__ long long s_off[2][TILE];  // a token's place in the cache, -1: none
  pdl_wait();
  pdl_trigger();
  tree_begin<kSimtRows, TILE, kSimtEnd>(A, &start, sums);
  auto walk = tree_walk<kSimtRows, TILE, kSimtEnd>(A, start);
  auto at = walk;
  const int tid = threadIdx.x, ty = tid / 16, tx = tid % 16;
  bool bad_page = false;

  while (walk.next(A, at)) {
    const TreeSpan& s = at.s;
    const int kvh = at.head(), r0 = at.block() * kSimtRows;
    const int rows = min(kSimtRows, s.use * A.group - r0);
    const float f = A.scale_log2;
    auto offsets = [&](int t, int buf) {
      if (tid >= TILE) return;
      const int pos = s.first + t * TILE + tid;
      long long off = -1;
      if (t < at.t1 && pos < s.len) {
        const int p = A.page_shift >= 0 ? pos >> A.page_shift : pos / A.page;
        const int id = __ldg(A.table + at.b * A.table_stride + p);
        if (id >= 0 && id < A.num_pages)
          off = id * A.s_page + (pos - p * A.page) * A.s_token + kvh * A.s_head;
      }
      s_off[buf][tid] = off;
    };
    auto load = [&](const char* base, float* to, int pitch, int buf) {
      constexpr int CPR = DP / 4;
      for (int i = tid; i < TILE * CPR; i += kSimtThreads) {
        const int r = i / CPR, c = i % CPR;
        const long long off = s_off[buf][r];
        const bool real = off >= 0 && c * 4 < A.dim;
        tree_cp16(smem_u32(to + r * pitch + c * 4), real ? base + off + c * 16 : base, real);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    offsets(at.t0, 0);
    for (int i = tid; i < kSimtRows * (DP / 4); i += kSimtThreads) {
      const int r = i / (DP / 4), d = i % (DP / 4) * 4;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < rows && d < A.dim) {
        const int R = r0 + r, node = R / A.group, h = kvh * A.group + R - node * A.group;
        v = *reinterpret_cast<const float4*>(static_cast<const float*>(A.q) +
                                             (s.row0 + node) * A.q_n + h * A.q_h + d);
      }
      *reinterpret_cast<float4*>(qs + r * KP + d) = v;
    }
    int node[2], low[2];
    TreeMask mask[2];
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f}, acc[2][4 * NC] = {};
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      node[e] = (r0 + min(2 * ty + e, rows - 1)) / A.group;
      mask[e] = tree_mask(A, s, node[e]);
      low[e] = tree_low(A, s, mask[e], node[e]);
    }
    __syncthreads();
    load(A.k, ks, KP, 0);
    load(A.v, vs, DP, 0);
    for (int t = at.t0; t < at.t1; ++t) {
      const int buf = (t - at.t0) & 1, pos0 = s.first + t * TILE;
      offsets(t + 1, buf ^ 1);
      asm volatile("cp.async.wait_group 1;" ::: "memory");
      __syncthreads();
      float x[2][NK] = {};
#pragma unroll 4
      for (int d = 0; d < DP; d += 4) {
        const float4 a = *reinterpret_cast<const float4*>(qs + (2 * ty) * KP + d);
        const float4 b = *reinterpret_cast<const float4*>(qs + (2 * ty + 1) * KP + d);
#pragma unroll
        for (int j = 0; j < NK; ++j) {
          const float4 k = *reinterpret_cast<const float4*>(ks + (tx + 16 * j) * KP + d);
          x[0][j] = fmaf(a.x, k.x, fmaf(a.y, k.y, fmaf(a.z, k.z, fmaf(a.w, k.w, x[0][j]))));
          x[1][j] = fmaf(b.x, k.x, fmaf(b.y, k.y, fmaf(b.z, k.z, fmaf(b.w, k.w, x[1][j]))));
        }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        unsigned live = 0;
        float top = -INFINITY;
#pragma unroll
        for (int j = 0; j < NK; ++j) {
          const int c = tx + 16 * j;
          const uint32_t bits = tree_attends(s, mask[e], low[e], pos0 + (c & ~31));
          bool on = bits >> (c & 31) & 1u;
          if (on && s_off[buf][c] < 0) {
            bad_page = true;
            on = false;
          }
          live |= static_cast<unsigned>(on) << j;
          x[e][j] *= f;
          if (on) top = fmaxf(top, x[e][j]);
        }
        if (live) top = fmaxf(top, -FLT_MAX);  // the row has tokens, if only of logits -inf
#pragma unroll
        for (int off = 8; off > 0; off >>= 1)
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
        const float to = fmaxf(m[e], top);
        const float keep = to == -INFINITY ? 1.0f : tree_ex2(m[e] - to);
        m[e] = to;
        l[e] *= keep;
#pragma unroll
        for (int c = 0; c < 4 * NC; ++c) acc[e][c] *= keep;
#pragma unroll
        for (int j = 0; j < NK; ++j) {
          const float p = live >> j & 1u ? tree_ex2(x[e][j] - to) : -1.0f;
          ps[(2 * ty + e) * PP + tx + 16 * j] = p;  // -1: not attended
          if (live >> j & 1u) l[e] += p;
        }
      }
      __syncthreads();
      load(A.k, ks, KP, buf ^ 1);
      asm volatile("cp.async.wait_group 1;" ::: "memory");
      __syncthreads();
#pragma unroll 2
      for (int c = 0; c < TILE; c += 4) {
        const float4 a4 = *reinterpret_cast<const float4*>(ps + (2 * ty) * PP + c);
        const float4 b4 = *reinterpret_cast<const float4*>(ps + (2 * ty + 1) * PP + c);
        const float pa[4] = {a4.x, a4.y, a4.z, a4.w}, pb[4] = {b4.x, b4.y, b4.z, b4.w};
#pragma unroll
        for (int u = 0; u < 4; ++u) {
#pragma unroll
          for (int j = 0; j < NC; ++j) {
            const float4 v = *reinterpret_cast<const float4*>(vs + (c + u) * DP + 4 * tx + 64 * j);
            if (!(pa[u] < 0.0f)) {
              acc[0][4 * j] = fmaf(pa[u], v.x, acc[0][4 * j]);
              acc[0][4 * j + 1] = fmaf(pa[u], v.y, acc[0][4 * j + 1]);
              acc[0][4 * j + 2] = fmaf(pa[u], v.z, acc[0][4 * j + 2]);
              acc[0][4 * j + 3] = fmaf(pa[u], v.w, acc[0][4 * j + 3]);
            }
            if (!(pb[u] < 0.0f)) {
              acc[1][4 * j] = fmaf(pb[u], v.x, acc[1][4 * j]);
              acc[1][4 * j + 1] = fmaf(pb[u], v.y, acc[1][4 * j + 1]);
              acc[1][4 * j + 2] = fmaf(pb[u], v.z, acc[1][4 * j + 2]);
              acc[1][4 * j + 3] = fmaf(pb[u], v.w, acc[1][4 * j + 3]);
            }
          }
        }
      }
      __syncthreads();
      load(A.v, vs, DP, buf ^ 1);
    }
    const bool whole = at.t0 == 0 && at.t1 == at.nt;
    const long long part = 2ll * blockIdx.x + (at.t0 == 0 ? 0 : 1);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
      for (int off = 8; off > 0; off >>= 1) l[e] += __shfl_xor_sync(0xffffffffu, l[e], off);
      const int r = 2 * ty + e;
      if (r >= rows) continue;
      if (whole) {
        const float inv = m[e] == -INFINITY ? 0.0f : 1.0f / l[e];
        const int R = r0 + r, h = kvh * A.group + R - node[e] * A.group;
        const long long row = s.row0 + node[e];
#pragma unroll
        for (int j = 0; j < NC; ++j)
          if (4 * tx + 64 * j < A.dim)
            tree_store4<MOE_KV_F32>(A.out, row * A.o_n + h * A.o_h + 4 * tx + 64 * j, acc[e][4 * j] * inv,
                            acc[e][4 * j + 1] * inv, acc[e][4 * j + 2] * inv,
                            acc[e][4 * j + 3] * inv);
        if (A.lse && tx == 0) A.lse[row * A.Hq + h] = tree_lse<MOE_KV_F32>(m[e], l[e]);
      } else {
#pragma unroll
        for (int j = 0; j < NC; ++j)
          *reinterpret_cast<float4*>(A.part_o + (part * kSimtRows + r) * DP + 4 * tx + 64 * j) =
              make_float4(acc[e][4 * j], acc[e][4 * j + 1], acc[e][4 * j + 2], acc[e][4 * j + 3]);
        if (tx == 0) A.part_ml[part * kSimtRows + r] = make_float2(m[e], l[e]);
      }
    }
    if (tid == 0 && at.t1 < at.nt) tree_record(A, start, at);
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();  // all of the tiles may be used again
  }
  if (bad_page && A.err) atomicOr(A.err, MOE_DEVERR_BAD_PAGE);
}

// ------------------------------------------------------------ host
struct TreeShape {
  int rows, tile, ctas_per_sm;
};
template <int DP>
static TreeShape shape_of(int kv) {
  if (kv == MOE_KV_F32) return {kSimtRows, SimtCfg<DP>::TILE, SimtCfg<DP>::CTAS};
  return {TcCfg<DP>::ROWS, TcCfg<DP>::TILE, TcCfg<DP>::CTAS};
}
static TreeShape tree_shape(int kv, int dp) {
  return dp == 64 ? shape_of<64>(kv) : dp == 128 ? shape_of<128>(kv) : shape_of<256>(kv);
}
static int tree_dp(int dim) { return dim <= 64 ? 64 : dim <= 128 ? 128 : 256; }

template <int DP>
static cudaError_t launch_simt(const TreeArgs& a, int ctas, cudaStream_t st) {
  auto* kern = tree_simt_kernel<DP>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), SimtCfg<DP>::SMEM, done);
  if (e != cudaSuccess) return e;
  e = launch_chained(kern, dim3(ctas), dim3(kSimtThreads), SimtCfg<DP>::SMEM, st, a);
  if (e != cudaSuccess) return e;
  return launch_chained(tree_join_kernel<MOE_KV_F32, DP, kSimtRows>, dim3(ctas, kTreeJoinBlocks),
                        dim3(32 * kTreeJoinWarps), 0, st, a);
}

static size_t up256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_attn_tree_workspace(int kv_dtype, int head_dim) {
  if (kv_dtype < MOE_KV_F32 || kv_dtype > MOE_KV_E4M3 || head_dim < 1 || head_dim > 256 ||
      head_dim % kv_dim_step(kv_dtype))
    return 0;
  const int dp = tree_dp(head_dim);
  const TreeShape s = tree_shape(kv_dtype, dp);
  const size_t n = static_cast<size_t>(sm_count()) * s.ctas_per_sm;
  return up256(n * sizeof(int4)) + up256(2 * n * s.rows * sizeof(float2)) +
         2 * n * s.rows * dp * sizeof(float);
}

int moe_attn_tree(const moe_kv_cache_t* cache, const void* q, long long q_stride_n,
                  long long q_stride_h, int N, int Hq, const int32_t* block_table, int max_pages,
                  long long table_stride, const int32_t* starts, const int32_t* seq_lens, int B,
                  const int64_t* masks, int max_new, float scale, int window, void* out,
                  long long o_stride_n, long long o_stride_h, float* lse, void* ws,
                  size_t ws_bytes, uint32_t* err, void* stream) {
  const int rc = kv_cache_ok(cache);
  if (rc != MOE_OK) return rc;
  if (N < 0 || B < 0 || Hq < 1 || Hq % cache->kv_heads || Hq > (1 << 20) ||
      static_cast<long long>(N) * Hq > INT_MAX || max_new < 1 || max_new > MOE_TREE_MAX ||
      max_pages < 1 || table_stride < max_pages || window < 0 ||
      static_cast<long long>(max_pages) * cache->page_size > INT_MAX - 1024 || q_stride_n < 0 ||
      q_stride_h < 0 || o_stride_n < 0 || o_stride_h < 0 || !std::isfinite(scale))
    return MOE_ERR_INVALID_ARG;
  if (B == 0 || N == 0) return MOE_OK;
  if (!q || !block_table || !starts || !seq_lens || !out || !ws) return MOE_ERR_INVALID_ARG;
  if (!apart(N, o_stride_n, cache->head_dim) || !apart(Hq, o_stride_h, cache->head_dim))
    return MOE_ERR_INVALID_ARG;
  const int qs = cache->kv_dtype == MOE_KV_F32 ? 4 : 2;
  if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(out) |
       static_cast<uintptr_t>(q_stride_n * qs) | static_cast<uintptr_t>(q_stride_h * qs) |
       static_cast<uintptr_t>(o_stride_n * qs) | static_cast<uintptr_t>(o_stride_h * qs)) &
      15)
    return MOE_ERR_UNSUPPORTED;
  if (reinterpret_cast<uintptr_t>(ws) & 255) return MOE_ERR_INVALID_ARG;
  if (ws_bytes < moe_attn_tree_workspace(cache->kv_dtype, cache->head_dim)) return MOE_ERR_WORKSPACE;
  const int sms = sm_count();
  if (sms < 1) return MOE_ERR_CUDA;
  const int es = kv_esize(cache->kv_dtype), dp = tree_dp(cache->head_dim);
  const TreeShape shape = tree_shape(cache->kv_dtype, dp);
  TreeArgs a = {};
  a.k = static_cast<const char*>(cache->k);
  a.v = static_cast<const char*>(cache->v);
  a.s_page = cache->stride_page * es;
  a.s_token = cache->stride_token * es;
  a.s_head = cache->stride_head * es;
  a.k_scale = cache->k_scale;
  a.v_scale = cache->v_scale;
  a.q = q;
  a.q_n = q_stride_n;
  a.q_h = q_stride_h;
  a.out = out;
  a.o_n = o_stride_n;
  a.o_h = o_stride_h;
  a.lse = lse;
  a.table = block_table;
  a.table_stride = table_stride;
  a.starts = starts;
  a.lens = seq_lens;
  a.masks = reinterpret_cast<const unsigned long long*>(masks);
  a.err = err;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.N = N;
  a.B = B;
  a.Hq = Hq;
  a.heads = cache->kv_heads;
  a.group = Hq / cache->kv_heads;
  a.words = (max_new + 63) / 64;
  a.max_new = max_new;
  a.dim = cache->head_dim;
  a.page = cache->page_size;
  a.page_shift = -1;
  for (int i = 0; i < 31; ++i)
    if (a.page == 1 << i) a.page_shift = i;
  a.num_pages = cache->num_pages;
  a.max_pages = max_pages;
  a.window = window;
  const int full = sms * shape.ctas_per_sm;
  uint8_t* w = static_cast<uint8_t*>(ws);
  a.info = reinterpret_cast<int4*>(w);
  w += up256(full * sizeof(int4));
  a.part_ml = reinterpret_cast<float2*>(w);
  w += up256(2ull * full * shape.rows * sizeof(float2));
  a.part_o = reinterpret_cast<float*>(w);
  // no more CTAs than (block, tile) pairs that these sizes can hold, whole groups
  const long long most = (static_cast<long long>(N < max_new ? N : max_new) * a.group +
                          shape.rows - 1) / shape.rows;
  const int size = static_cast<int>(most < kTreeGroup ? most : kTreeGroup);
  const long long tiles = (static_cast<long long>(max_pages) * a.page + shape.tile - 1) / shape.tile;
  const long long units = (B < N ? B : N) * ((most + size - 1) / size) * a.heads;
  const int ctas = units >= full || tiles >= full || units * tiles * size >= full
                       ? full
                       : static_cast<int>(units * tiles) * size;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = cache->kv_dtype != MOE_KV_F32 ? launch_tree_tc(cache->kv_dtype, dp, a, ctas, st)
                        : dp == 64                    ? launch_simt<64>(a, ctas, st)
                        : dp == 128                   ? launch_simt<128>(a, ctas, st)
                                                      : launch_simt<256>(a, ctas, st);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
