// adjust.cu -- penalties for repeated tokens, biases and allowed tokens applied
// to logits before a token is drawn (moe_adjust_logits).
//
// One pass over the logits: each is read once and written once.  A CTA has a slice
// of a row.  What a token's logit needs to know of the request's history is a word
// in shared memory, bit 31: it occurs, below: how often in the answer; every CTA
// of a row reads the history for itself and counts the tokens of its slice, while
// its logits are on their way.  (The CTAs of a row as a cluster that deals the
// history out and counts in each other's memory: 205 us for 512 rows of 131072,
// f32; a text's frequent tokens make remote additions queue up.)  Counts are
// whole numbers: the order of additions does not show.  At a node of a tree the
// drafted tokens on its path count too, a node a thread: 3% more (16 requests x 64
// nodes of 131072, bf16: 161 us instead of 155).
//
// Biases are few: their tokens are adjusted once more behind the pass, from logits
// that were set aside before it.  (A place in the list for every token of the slice
// in shared memory: 139 us for the same rows.)
//
// Bound by the logits' bytes without a history (512 rows of 131072, f32: 78 us, 6.9
// TB/s, as long as a copy takes); with histories of up to 8192 tokens, a hundred
// biases and masks 120 us, 4.6 TB/s: the chain from lengths to tokens to counts,
// and each CTA's own pass over the history, are longer than its loads take.  64
// rows of 50257, bf16: 9.7 us, that chain.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>

#include "../../include/moe_route.h"
#include "decode_internal.cuh"
#include "moe_internal.cuh"
#include "ptx.cuh"

namespace moe {

constexpr int kAdjustThreads = 256;
constexpr int kAdjustSlice = 8192;  // tokens of a CTA at most
constexpr int kAdjustBias = MOE_ADJUST_MAX_BIAS;

struct AdjustArgs {
  const char* x;
  char* out;
  long long x_row, out_row;  // elements
  const int* rows;           // NULL: row i is request i
  const int* history;
  long long history_stride;
  const int *history_lens, *prompt_lens;
  const float *repetition, *presence, *frequency;
  const int* bias_ids;
  const float* bias;
  const unsigned* allowed;
  long long allowed_stride;  // words
  const int* tokens;         // NULL: no drafted tokens
  const unsigned long long* masks;
  const int* starts;
  unsigned* err;
  int N, V, R, max_history, n_bias, mask_words;
  int slice;  // tokens of a CTA, a multiple of 32
};

template <typename T>
__device__ __forceinline__ float as_f32(T v);
template <>
__device__ __forceinline__ float as_f32<float>(float v) {
  return v;
}
template <>
__device__ __forceinline__ float as_f32<__nv_bfloat16>(__nv_bfloat16 v) {
  return __bfloat162float(v);
}
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) {
  return v;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

// PAST: a history (or drafted tokens) with penalties; BIAS: a list of biases
template <typename T, bool PAST, bool BIAS>
__global__ void __launch_bounds__(kAdjustThreads, 4) adjust_kernel(const AdjustArgs A) {
  extern __shared__ uint4 adjust_smem[];
  constexpr int VE = 16 / sizeof(T);
  constexpr int U = kAdjustSlice / kAdjustThreads / VE;  // vectors of a thread
  pdl_wait();
  const int tid = threadIdx.x;
  const int row = blockIdx.y, lo = blockIdx.x * A.slice;
  const int n = max(0, min(A.slice, A.V - lo));
  const T* const x = reinterpret_cast<const T*>(A.x) + row * A.x_row + lo;
  T* const out = reinterpret_cast<T*>(A.out) + row * A.out_row + lo;
  // the slice's tokens before the first 16-byte boundary of the logits; the words
  // are shifted so that a vector of logits has a vector of words
  const int skew = static_cast<int>(reinterpret_cast<uintptr_t>(x) / sizeof(T) % VE);
  uint32_t* const words = reinterpret_cast<uint32_t*>(adjust_smem) + skew;
  // the logits are asked for before anything else: they arrive while the history
  // is counted
  const int head = min(n, (VE - skew) % VE), vecs = (n - head) / VE, tail = head + vecs * VE;
  uint4 raw[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int i = u * kAdjustThreads + tid;
    if (i < vecs) raw[u] = __ldcs(reinterpret_cast<const uint4*>(x + head + i * VE));
  }
  int req = A.rows ? A.rows[row] : row;
  if (req < 0 || req >= A.R) {
    if (A.err && blockIdx.x == 0 && tid == 0) atomicOr(A.err, MOE_DEVERR_BAD_ID);
    req = -1;
  }
  // the slice's words of allowed tokens and the list of biased ones go to shared
  // memory; asked for here as well
  __shared__ uint32_t s_allowed[kAdjustSlice / 32];
  __shared__ int s_ids[BIAS ? kAdjustBias : 1];
  static_assert(kAdjustSlice / 32 == kAdjustThreads, "a word a thread");
  const unsigned* const allowed = A.allowed ? A.allowed + row * A.allowed_stride : nullptr;
  uint32_t my_allowed = ~0u;
  if (allowed && 32 * tid < n) my_allowed = __ldg(allowed + lo / 32 + tid);
  constexpr int K = BIAS ? kAdjustBias / kAdjustThreads : 1;  // biases of a thread at most
  const int n_bias = BIAS && req >= 0 ? A.n_bias : 0;
  int id[K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int j = k * kAdjustThreads + tid;
    id[k] = -1;
    if (j < n_bias) id[k] = __ldg(A.bias_ids + static_cast<long long>(req) * A.n_bias + j);
  }
  float rep = 1.0f, freq = 0.0f, pres = 0.0f;
  constexpr int AT_ONCE = 8;  // tokens of the history that a thread asks for
  int len = 0, prompt = 0, past[AT_ONCE], drafted = -1;
  const int* h = nullptr;
  auto ask = [&](long long i0) {
#pragma unroll
    for (int u = 0; u < AT_ONCE; ++u) {
      const long long i = i0 + u * kAdjustThreads;
      past[u] = i < len ? __ldg(h + i) : -1;
    }
  };
  if (PAST && req >= 0) {
    if (A.repetition) rep = A.repetition[req];
    if (A.presence) pres = A.presence[req];
    if (A.frequency) freq = A.frequency[req];
    if (A.max_history > 0) len = max(0, min(A.history_lens[req], A.max_history));
    prompt = A.prompt_lens ? A.prompt_lens[req] : 0;
    h = A.history + req * A.history_stride;
    ask(tid);
    if (A.tokens && tid > 0) {  // node tid, if the row attends it
      static_assert(MOE_TREE_MAX <= kAdjustThreads, "a node a thread");
      const int row0 = max(0, min(A.starts[req], A.N)), end = min(A.starts[req + 1], A.N);
      if (row >= row0 && row < end && row0 + tid < end && tid < 64 * A.mask_words &&
          A.masks[static_cast<long long>(row) * A.mask_words + tid / 64] >> (tid % 64) & 1)
        drafted = A.tokens[row0 + tid];
    }
  }
  if constexpr (PAST) {
    const int w16 = (A.slice + VE) / 4;
    for (int i = tid; i < w16; i += kAdjustThreads) adjust_smem[i] = make_uint4(0, 0, 0, 0);
  }
  s_allowed[tid] = my_allowed;
  if constexpr (BIAS) {
#pragma unroll
    for (int k = 0; k < K; ++k) s_ids[k * kAdjustThreads + tid] = id[k];
  }
  __syncthreads();
  if constexpr (PAST) {
    for (long long i0 = tid; i0 < len; i0 += AT_ONCE * kAdjustThreads) {
      if (i0 > tid) ask(i0);
#pragma unroll
      for (int u = 0; u < AT_ONCE; ++u) {
        if (past[u] < lo || past[u] - lo >= n) continue;
        if (i0 + u * kAdjustThreads < prompt) atomicOr(words + (past[u] - lo), 0x80000000u);
        else atomicAdd(words + (past[u] - lo), 1u);
      }
    }
    if (drafted >= lo && drafted - lo < n) atomicAdd(words + (drafted - lo), 1u);
  }
  // a biased token of the slice: its logit and its bias, for later.  Of equal ids the
  // last counts
  float biased[K], more[K];
  if constexpr (BIAS) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int j = k * kAdjustThreads + tid;
      if (id[k] < lo || id[k] - lo >= n) id[k] = -1;
      if (id[k] < 0) continue;
      for (int i = j + 1; i < n_bias; ++i)
        if (s_ids[i] == id[k]) id[k] = -1;
      if (id[k] < 0) continue;
      biased[k] = as_f32<T>(x[id[k] - lo]);
      more[k] = __ldg(A.bias + static_cast<long long>(req) * A.n_bias + j);
    }
  }
  if constexpr (PAST || BIAS) __syncthreads();

  auto adjust = [&](float v, uint32_t word, float add, bool ok) {
    if constexpr (PAST) {
      if (word) {
        v = v > 0.0f ? v / rep : v * rep;
        const uint32_t c = word & 0x7fffffffu;
        v -= freq * static_cast<float>(c);
        if (c) v -= pres;
      }
    }
    if constexpr (BIAS) v += add;
    return ok ? v : -INFINITY;
  };
  auto one = [&](int t) {
    const float v = as_f32<T>(x[t]);
    const bool ok = s_allowed[t / 32] >> (t & 31) & 1u;
    out[t] = from_f32<T>(adjust(v, PAST ? words[t] : 0u, 0.0f, ok));
  };
  const bool same = reinterpret_cast<uintptr_t>(out) / sizeof(T) % VE == static_cast<unsigned>(skew);
  if (tid < head) one(tid);
  if (tail + tid < n) one(tail + tid);
  {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = u * kAdjustThreads + tid;
      if (i >= vecs) break;
      const int t = head + i * VE;
      T* const v = reinterpret_cast<T*>(raw + u);
      constexpr unsigned ALL = (1u << VE) - 1;
      auto bits_of = [&](const uint32_t* map) {  // VE tokens may lie in two words
        const int k = t / 32, s = t & 31;
        unsigned bits = map[k] >> s;
        if (s > 32 - VE) bits |= map[k + 1] << (32 - s);
        return bits & ALL;
      };
      const unsigned ok = allowed ? bits_of(s_allowed) : ALL;
      uint4 w[VE / 4];
      uint32_t touched = 0;
#pragma unroll
      for (int j = 0; j < VE / 4; ++j) {
        w[j] = make_uint4(0, 0, 0, 0);
        if constexpr (PAST) w[j] = *reinterpret_cast<const uint4*>(words + t + 4 * j);
        touched |= w[j].x | w[j].y | w[j].z | w[j].w;
      }
      if (touched) {  // few are
#pragma unroll
        for (int j = 0; j < VE; ++j) {
          const uint4 a = w[j / 4];
          const uint32_t word = j % 4 == 0 ? a.x : j % 4 == 1 ? a.y : j % 4 == 2 ? a.z : a.w;
          v[j] = from_f32<T>(adjust(as_f32<T>(v[j]), word, 0.0f, ok >> j & 1u));
        }
      } else if (ok != ALL) {
#pragma unroll
        for (int j = 0; j < VE; ++j)
          if (!(ok >> j & 1u)) v[j] = from_f32<T>(-INFINITY);
      }
      if (same) {
        __stcs(reinterpret_cast<uint4*>(out + t), raw[u]);
      } else {
#pragma unroll
        for (int j = 0; j < VE; ++j) out[t + j] = v[j];
      }
    }
  }
  if constexpr (BIAS) {  // the biased ones once more
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (id[k] < 0) continue;
      const int t = id[k] - lo;
      const bool ok = s_allowed[t / 32] >> (t & 31) & 1u;
      out[t] = from_f32<T>(adjust(biased[k], PAST ? words[t] : 0u, more[k], ok));
    }
  }
}

template <typename T, bool PAST, bool BIAS>
static cudaError_t launch_adjust(AdjustArgs a, cudaStream_t st) {
  auto* kern = adjust_kernel<T, PAST, BIAS>;
  const int ve = 16 / sizeof(T);
  // few rows: smaller slices, until every SM has one
  a.slice = kAdjustSlice;
  while (a.slice > 1024 && static_cast<long long>(a.N) * ((a.V - 1) / a.slice + 1) < sm_count())
    a.slice /= 2;
  const int smem = PAST ? (a.slice + ve) * 4 : 0;
  static std::atomic<uint64_t> done{0};
  if (smem > 0) {
    const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern),
                                     (kAdjustSlice + ve) * 4, done);
    if (e != cudaSuccess) return e;
  }
  return launch_chained(kern, dim3((a.V - 1) / a.slice + 1, a.N), dim3(kAdjustThreads), smem, st, a);
}

template <typename T>
static cudaError_t launch_type(const AdjustArgs& a, cudaStream_t st) {
  const bool past = a.max_history > 0 || a.tokens;
  if (past) return a.n_bias > 0 ? launch_adjust<T, true, true>(a, st) : launch_adjust<T, true, false>(a, st);
  return a.n_bias > 0 ? launch_adjust<T, false, true>(a, st) : launch_adjust<T, false, false>(a, st);
}

}  // namespace moe

using namespace moe;

extern "C" int moe_adjust_logits(const moe_adjust_t* s, const void* logits, int logits_dtype, int N,
                                 int V, long long row_stride, void* out, long long out_stride,
                                 uint32_t* err, void* stream) {
  if (!s || N < 0 || N > 65535 || V < 1 || V > (1 << 18) || row_stride < 0 ||
      (logits_dtype != MOE_LOGITS_F32 && logits_dtype != MOE_LOGITS_BF16) || s->requests < 0 ||
      s->max_history < 0 || s->n_bias < 0 || s->n_bias > MOE_ADJUST_MAX_BIAS || s->history_stride < 0 ||
      s->allowed_stride < 0)
    return MOE_ERR_INVALID_ARG;
  if (!s->rows && s->requests < N) return MOE_ERR_INVALID_ARG;
  if (N == 0) return MOE_OK;
  const int es = logits_dtype == MOE_LOGITS_F32 ? 4 : 2;
  if (!logits || !out || !apart(N, out_stride, V)) return MOE_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(logits) | reinterpret_cast<uintptr_t>(out)) & (es - 1))
    return MOE_ERR_INVALID_ARG;
  if (s->history && s->max_history > 0 && !s->history_lens) return MOE_ERR_INVALID_ARG;
  if (s->n_bias > 0 && (!s->bias_ids || !s->bias)) return MOE_ERR_INVALID_ARG;
  if (s->mask_words < 0 || s->mask_words > MOE_TREE_MAX / 64 ||
      (s->mask_words > 0 && (!s->tokens || !s->masks || !s->starts)))
    return MOE_ERR_INVALID_ARG;
  // the logits themselves may be the output; anything else must not overlap them
  const uintptr_t x0 = reinterpret_cast<uintptr_t>(logits), o0 = reinterpret_cast<uintptr_t>(out);
  const uintptr_t x1 = x0 + (static_cast<uintptr_t>(N - 1) * row_stride + V) * es;
  const uintptr_t o1 = o0 + (static_cast<uintptr_t>(N - 1) * out_stride + V) * es;
  const bool itself = x0 == o0 && (N == 1 || row_stride == out_stride);
  if (!itself && x0 < o1 && o0 < x1) return MOE_ERR_INVALID_ARG;
  AdjustArgs a = {};
  a.x = static_cast<const char*>(logits);
  a.out = static_cast<char*>(out);
  a.x_row = row_stride;
  a.out_row = out_stride;
  a.rows = s->rows;
  a.history = s->history;
  a.history_stride = s->history_stride;
  a.history_lens = s->history_lens;
  a.prompt_lens = s->prompt_lens;
  a.repetition = s->repetition;
  a.presence = s->presence;
  a.frequency = s->frequency;
  a.bias_ids = s->bias_ids;
  a.bias = s->bias;
  a.allowed = reinterpret_cast<const unsigned*>(s->allowed);
  a.allowed_stride = s->allowed_stride;
  a.err = err;
  a.N = N;
  a.V = V;
  a.R = s->requests;
  a.max_history = s->history ? s->max_history : 0;
  if (s->mask_words > 0) {
    a.tokens = s->tokens;
    a.masks = reinterpret_cast<const unsigned long long*>(s->masks);
    a.starts = s->starts;
    a.mask_words = s->mask_words;
  }
  a.n_bias = s->n_bias;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = logits_dtype == MOE_LOGITS_F32 ? launch_type<float>(a, st)
                                                       : launch_type<__nv_bfloat16>(a, st);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
