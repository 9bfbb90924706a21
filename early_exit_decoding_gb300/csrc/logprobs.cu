// Log-probabilities of given tokens, entropy and top alternatives of rows of
// logits (rl_token_logprobs).
//
// With m = max x and s = sum exp(x - m):  lse = m + ln s,
// entropy = ln s - (sum (x - m) exp(x - m)) / s,  logprob_t = (x_t - m) - ln s.
//
// Simplest form: one CTA per row, one pass for the maximum, one for the two
// sums, one per alternative.
#include <float.h>

#include "dev_common.cuh"
#include "internal.h"

namespace river {

namespace {

using namespace dev;

constexpr int kThreads = 256;

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(bf16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }

// Unsigned keys that order values as documented: NaN above +infinity, -0 as
// +0; the low half orders equal values by the lower id.
__device__ __forceinline__ unsigned long long order_key(float x, int id) {
  uint32_t u = x != x ? 0x7fffffffu : __float_as_uint(x + 0.f);
  u = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
  return ((unsigned long long)u << 32) | (0xffffffffu - (uint32_t)id);
}
__device__ __forceinline__ unsigned long long warp_max_u64(unsigned long long v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const unsigned long long w = __shfl_xor_sync(0xffffffffu, v, o);
    v = w > v ? w : v;
  }
  return v;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) k_logprobs_rows(LogprobArgs a) {
  __shared__ float sf[3][kThreads / 32];
  __shared__ unsigned long long sk[kThreads / 32];
  const int r = blockIdx.x, tid = threadIdx.x, w = tid >> 5, l = tid & 31;
  const T* x = static_cast<const T*>(a.x) + (long long)r * a.ld;
  float m = -INFINITY;
  bool bad = false;
  for (int i = tid; i < a.V; i += kThreads) {
    const float v = to_f(x[i]);
    bad |= v != v;
    m = fmaxf(m, v);
  }
  m = warp_max(m);
  if (l == 0) sf[0][w] = m;
  bad = __syncthreads_or(bad);
  m = sf[0][0];
  for (int i = 1; i < kThreads / 32; ++i) m = fmaxf(m, sf[0][i]);
  __syncthreads();
  float s = 0.f, t = 0.f;
  for (int i = tid; i < a.V; i += kThreads) {
    const float d = fmaxf(to_f(x[i]) - m, -1e30f), e = __expf(d);
    s += e;
    t += d * e;
  }
  s = warp_sum(s);
  t = warp_sum(t);
  if (l == 0) {
    sf[1][w] = s;
    sf[2][w] = t;
  }
  __syncthreads();
  s = t = 0.f;
  for (int i = 0; i < kThreads / 32; ++i) {
    s += sf[1][i];
    t += sf[2][i];
  }
  const bool none = m == -INFINITY && !bad;
  if (bad || m == INFINITY) s = NAN;
  const float ln_s = none ? NAN : logf(s);
  if (tid == 0) {
    if (a.lse) a.lse[r] = none ? -INFINITY : m + ln_s;
    if (a.entropy) a.entropy[r] = ln_s - t / s;
  }
  for (int i = tid; i < a.n_tok; i += kThreads) {
    const int tok = a.tokens[(long long)r * a.n_tok + i];
    float v = NAN;
    if (tok >= 0 && tok < a.V)
      v = (to_f(x[tok]) - m) - ln_s;
    else if (a.err)
      atomicOr(a.err, RL_DEVERR_TOKEN);
    a.logprob[(long long)r * a.n_tok + i] = v;
  }
  unsigned long long last = ~0ull;
  for (int k = 0; k < a.top_k; ++k) {
    unsigned long long best = 0;
    for (int i = tid; i < a.V; i += kThreads) {
      const unsigned long long key = order_key(to_f(x[i]), i);
      if (key < last && key > best) best = key;
    }
    best = warp_max_u64(best);
    if (l == 0) sk[w] = best;
    __syncthreads();
    for (int i = 0; i < kThreads / 32; ++i) best = sk[i] > best ? sk[i] : best;
    __syncthreads();
    last = best;
    if (tid == 0) {
      const int id = (int)(0xffffffffu - (uint32_t)best);
      a.top_ids[(long long)r * a.top_k + k] = id;
      a.top_lp[(long long)r * a.top_k + k] = (to_f(x[id]) - m) - ln_s;
    }
  }
}

}  // namespace

cudaError_t launch_logprobs(const LogprobArgs& a, cudaStream_t s) {
  if (a.dtype == RL_DT_F32)
    k_logprobs_rows<float><<<a.rows, kThreads, 0, s>>>(a);
  else if (a.dtype == RL_DT_BF16)
    k_logprobs_rows<bf16><<<a.rows, kThreads, 0, s>>>(a);
  else
    k_logprobs_rows<__half><<<a.rows, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace river

using namespace river;

extern "C" rl_status rl_token_logprobs(const void* d_logits, int32_t dtype, int32_t rows, int32_t vocab,
                                       int64_t row_stride, const int32_t* d_tokens, int32_t n_tok,
                                       int32_t top_k, float* d_lse, float* d_entropy, float* d_logprob,
                                       int32_t* d_top_ids, float* d_top_logprobs, int32_t* d_err,
                                       rl_stream_t stream) {
  if (!d_logits) return set_error(RL_ERR_INVALID_ARG, "rl_token_logprobs: logits are NULL");
  if (dtype != RL_DT_F32 && dtype != RL_DT_BF16 && dtype != RL_DT_F16)
    return set_error(RL_ERR_INVALID_ARG, "rl_token_logprobs: unknown dtype");
  if (rows < 1 || vocab < 1 || row_stride < vocab)
    return set_error(RL_ERR_INVALID_ARG, "rl_token_logprobs: rows and vocab must be >= 1, row_stride >= vocab");
  if (n_tok < 0 || n_tok > 256 || (n_tok > 0 && (!d_tokens || !d_logprob)))
    return set_error(RL_ERR_INVALID_ARG, "rl_token_logprobs: n_tok outside [0, 256], or tokens or logprob NULL");
  if (top_k < 0 || top_k > 32 || top_k > vocab || (top_k > 0 && (!d_top_ids || !d_top_logprobs)))
    return set_error(RL_ERR_INVALID_ARG, "rl_token_logprobs: top_k outside [0, min(32, vocab)], or its outputs NULL");
  const size_t es = dtype == RL_DT_F32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(d_logits) % es)
    return set_error(RL_ERR_INVALID_ARG, "rl_token_logprobs: logits off their element's alignment");
  LogprobArgs a = {};
  a.x = d_logits;
  a.dtype = dtype;
  a.rows = rows;
  a.V = vocab;
  a.ld = row_stride;
  a.tokens = d_tokens;
  a.n_tok = n_tok;
  a.top_k = top_k;
  a.lse = d_lse;
  a.entropy = d_entropy;
  a.logprob = d_logprob;
  a.top_ids = d_top_ids;
  a.top_lp = d_top_logprobs;
  a.err = d_err;
  const cudaError_t e = launch_logprobs(a, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return set_error(RL_ERR_CUDA, cudaGetErrorString(e));
  return RL_OK;
}
