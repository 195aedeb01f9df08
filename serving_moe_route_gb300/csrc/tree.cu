// tree.cu -- trees of drafted tokens: which tokens each of them attends
// (moe_tree_masks), and which of them the tokens drawn at them accept
// (moe_tree_accept).  One CTA per request; a request's nodes are in shared
// memory, where all chains of dependent steps run.  Bound by latency: lengths,
// nodes, and a step per level.  128 requests of 64 nodes, caches cold: 4.9 us for
// the masks, 5.0 for the walk; the host's calls take 4.1 and 4.7.
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>

#include "../../include/moe_route.h"
#include "decode_internal.cuh"
#include "moe_internal.cuh"
#include "ptx.cuh"

namespace moe {

constexpr int kTreeThreads = 128;
constexpr int kTreeWords = MOE_TREE_MAX / 64;

// rows [x, y) of request r: inside [0, N), and none where starts does not rise
__device__ __forceinline__ int2 rows_of(const int* starts, int r, int N) {
  const int lo = max(0, min(starts[r], N));
  return make_int2(lo, max(lo, min(starts[r + 1], N)));
}

struct MaskArgs {
  const int *parents, *starts, *lens;
  unsigned long long* masks;  // [N][words]
  int* positions;
  unsigned* err;
  int N, B, words, max_new;
};

// A node's mask is its own bit and its parent's mask.  The distance looked up
// doubles from round to round, so the deepest chain of 256 takes 8.
__global__ void __launch_bounds__(kTreeThreads) tree_masks_kernel(const MaskArgs A) {
  __shared__ unsigned long long s_mask[2][kTreeWords][MOE_TREE_MAX];
  __shared__ short s_up[2][MOE_TREE_MAX];
  pdl_wait();
  const int tid = threadIdx.x, r = blockIdx.x;
  const int2 rows = rows_of(A.starts, r, A.N);
  const int n = min(rows.y - rows.x, A.max_new);
  unsigned bad = rows.y - rows.x > n ? MOE_DEVERR_NO_SPACE : 0;
  for (int j = tid; j < n; j += kTreeThreads) {
    int up = A.parents[rows.x + j];
    if (up < -1 || up >= j) {
      bad |= MOE_DEVERR_BAD_ID;
      up = -1;
    }
    s_up[0][j] = static_cast<short>(up);
    for (int w = 0; w < A.words; ++w) s_mask[0][w][j] = w == j / 64 ? 1ull << (j % 64) : 0;
  }
  __syncthreads();
  int at = 0;
  for (int reach = 1; reach < n; reach *= 2) {
    for (int j = tid; j < n; j += kTreeThreads) {
      const int up = s_up[at][j];
      for (int w = 0; w < A.words; ++w)
        s_mask[at ^ 1][w][j] = s_mask[at][w][j] | (up >= 0 ? s_mask[at][w][up] : 0);
      s_up[at ^ 1][j] = up >= 0 ? s_up[at][up] : -1;
    }
    at ^= 1;
    __syncthreads();
  }
  const int ctx = max(0, max(0, A.lens[r]) - (rows.y - rows.x));
  for (int j = tid; j < rows.y - rows.x; j += kTreeThreads) {
    int depth = 0;
    for (int w = 0; w < A.words; ++w) {
      const unsigned long long m = j < n ? s_mask[at][w][j] : 0;
      A.masks[static_cast<long long>(rows.x + j) * A.words + w] = m;
      depth += __popcll(m);
    }
    A.positions[rows.x + j] = ctx + max(0, depth - 1);
  }
  // rows of no request
  const int end = rows_of(A.starts, A.B - 1, A.N).y, head = rows_of(A.starts, 0, A.N).x;
  const int idle = head + A.N - end;
  for (long long i = static_cast<long long>(r) * kTreeThreads + tid; i < idle;
       i += static_cast<long long>(A.B) * kTreeThreads) {
    const long long row = i < head ? i : end + (i - head);
    for (int w = 0; w < A.words; ++w) A.masks[row * A.words + w] = 0;
    A.positions[row] = 0;
  }
  if (bad && A.err) atomicOr(A.err, bad);
}

struct AcceptArgs {
  const int *tokens, *draws, *parents, *starts, *ctx;
  int *path, *accepted, *next, *lens;
  unsigned* err;
  int N, max_path;
};

// Every node looks whether it is the token drawn at its parent; the parent keeps
// the lowest such child, and the walk is a chain through shared memory.
__global__ void __launch_bounds__(kTreeThreads) tree_accept_kernel(const AcceptArgs A) {
  __shared__ int s_child[MOE_TREE_MAX];
  pdl_wait();
  const int tid = threadIdx.x, r = blockIdx.x;
  const int2 rows = rows_of(A.starts, r, A.N);
  const int n = min(rows.y - rows.x, MOE_TREE_MAX);
  unsigned bad = rows.y - rows.x > n ? MOE_DEVERR_NO_SPACE : 0;
  for (int j = tid; j < n; j += kTreeThreads) s_child[j] = INT_MAX;
  __syncthreads();
  for (int j = tid; j < n; j += kTreeThreads) {
    const int up = A.parents[rows.x + j];
    if (up < -1 || up >= j) {
      bad |= MOE_DEVERR_BAD_ID;
    } else if (up >= 0) {
      const int draw = A.draws[rows.x + up];
      if (draw >= 0 && draw == A.tokens[rows.x + j]) atomicMin(s_child + up, j);
    }
  }
  __syncthreads();
  int* const path = A.path + static_cast<long long>(r) * A.max_path;
  if (tid == 0) {
    int count = 0, last = -1;
    for (int cur = n > 0 ? 0 : INT_MAX; cur != INT_MAX && count < A.max_path; cur = s_child[cur]) {
      path[count++] = cur;
      last = cur;
    }
    A.accepted[r] = count;
    A.next[r] = last >= 0 ? A.draws[rows.x + last] : -1;
    A.lens[r] = min(max(0, A.ctx[r]), INT_MAX - count) + count;
    s_child[0] = count;  // (the walk is over)
  }
  __syncthreads();
  for (int j = s_child[0] + tid; j < A.max_path; j += kTreeThreads) path[j] = -1;
  if (bad && A.err) atomicOr(A.err, bad);
}

}  // namespace moe

using namespace moe;

extern "C" {

int moe_tree_masks(const int32_t* parents, int N, const int32_t* starts, const int32_t* seq_lens,
                   int B, int max_new, int64_t* masks, int32_t* positions, uint32_t* err,
                   void* stream) {
  if (N < 0 || B < 0 || max_new < 1 || max_new > MOE_TREE_MAX || (B == 0 && N > 0))
    return MOE_ERR_INVALID_ARG;
  if (B == 0) return MOE_OK;
  if (!starts || !seq_lens || (N > 0 && (!parents || !masks || !positions)))
    return MOE_ERR_INVALID_ARG;
  const MaskArgs a = {parents, starts, seq_lens, reinterpret_cast<unsigned long long*>(masks),
                      positions, err, N, B, (max_new + 63) / 64, max_new};
  return launch_chained(tree_masks_kernel, dim3(B), dim3(kTreeThreads), 0,
                        static_cast<cudaStream_t>(stream), a) == cudaSuccess
             ? MOE_OK
             : MOE_ERR_CUDA;
}

int moe_tree_accept(const int32_t* tokens, const int32_t* draws, const int32_t* parents, int N,
                    const int32_t* starts, const int32_t* ctx_lens, int B, int max_path,
                    int32_t* path, int32_t* accepted, int32_t* next_ids, int32_t* seq_lens,
                    uint32_t* err, void* stream) {
  if (N < 0 || B < 0 || max_path < 1 || max_path > MOE_TREE_MAX) return MOE_ERR_INVALID_ARG;
  if (B == 0) return MOE_OK;
  if (!starts || !ctx_lens || !path || !accepted || !next_ids || !seq_lens ||
      (N > 0 && (!tokens || !draws || !parents)))
    return MOE_ERR_INVALID_ARG;
  const AcceptArgs a = {tokens, draws, parents, starts, ctx_lens, path, accepted, next_ids,
                        seq_lens, err, N, max_path};
  return launch_chained(tree_accept_kernel, dim3(B), dim3(kTreeThreads), 0,
                        static_cast<cudaStream_t>(stream), a) == cudaSuccess
             ? MOE_OK
             : MOE_ERR_CUDA;
}

}  // extern "C"
