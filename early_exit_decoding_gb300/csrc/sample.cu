// Sampling from rows of logits with temperature, top-k, top-p and min-p, by a
// given random number (rl_sample).
//
// The ids ordered by (logit, lower id) are kept up to some last one, so what the
// three filters keep is a key: ids whose 64-bit key (ordered logit, then the
// lower id) is at least `cut`.  top-k's cut is the k-th largest key, top-p's the
// key at which the weights' running sum reaches top_p of their total, both
// found a digit of the key at a time (a histogram of the ids that agree in the
// digits before: counts, or weights); min-p's is a logit.  The token is then
// found among the ids of at least `cut` by running sums in the order of ids.
//
// A weight is a 64-bit whole number, exp((x - max) / T) 2^44 rounded: sums are
// exact whatever their order, and with exponentials good to 2^-38 a token
// differs from that of exact weights only where u is that near a border (fp32
// sums: 1 in 50 rows of 128,256 logits with a long tail).
//
// Simplest form: one CTA a row, which reads the row once a step.
#include <float.h>
#include <math.h>
#include <stdio.h>

#include "dev_common.cuh"
#include "internal.h"

namespace river {

struct SampleArgs {
  const void* x;
  int dtype, rows, V;
  long long ld;
  const float* u;
  rl_sampling set;
  int* token;
  float* logprob;
  int* err;
};

namespace {

using namespace dev;
using u64 = unsigned long long;

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;

__device__ __forceinline__ uint32_t order_bits(float x) {
  const uint32_t u = x != x ? 0x7fffffffu : __float_as_uint(x + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t o) {
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7fffffffu) : ~o);
}
__device__ __forceinline__ u64 key_of(float x, int id) { return ((u64)order_bits(x) << 32) | (0xffffffffu - (uint32_t)id); }

// 2^(-j / 64) 2^44, j < 64.
struct Pow2Table {
  u64 t[64];
};

// exp((x - m) / T) 2^44, rounded: 2^-y with y = (m - x) c, c = log2(e) / T.
struct Weight {
  float m, ch, cl;  // c = ch + cl
  const u64* table;
  __device__ __forceinline__ u64 operator()(float x) const {
    // y = p + e: the difference and the product exact in two parts each
    const float d = m - x, b = d - m, dl = (m - (d - b)) - (x + b);
    const float p = d * ch;
    if (!(p < 46.f)) return 0;  // (below half a unit; x = -infinity, or c 0 times infinity)
    const float e = fmaf(dl, ch, fmaf(d, cl, fmaf(d, ch, -p)));
    // y = k / 64 + r, |r| <= 1 / 128
    const float big = 196608.f;  // 1.5 2^17: its sums are whole multiples of 1 / 64
    const float s = p + big, r = p - (s - big);
    const int k = (int)(__float_as_uint(s) - __float_as_uint(big));
    // 2^-r = 1 - a + a^2 / 2 - a^3 / 6 + a^4 / 24 (the next term is below 2^-44), a = ln 2 (r + e) = ah + al
    const float lh = 0.693147182464599609375f, ll = -1.904654323148236017e-9f;  // ln 2 in two parts
    const float ah = r * lh, al = fmaf(e, lh, fmaf(r, ll, fmaf(r, lh, -ah)));
    const float v = fmaf(-ah * ah, fmaf(ah, fmaf(ah, 1.f / 24.f, -1.f / 6.f), 0.5f), al);  // 1 - 2^-r = ah + v
    const long long w = (long long)__float2int_rn(ah * 274877906944.f) + __float2int_rn(v * 274877906944.f);  // 2^38
    const u64 t = table[k & 63];
    const int n = k >> 6;
    const u64 f = t - (u64)(((long long)(t >> 13) * w) >> 25);
    return (f + ((1ull << n) >> 1)) >> n;
  }
};

__device__ __forceinline__ u64 warp_sum64(u64 v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <typename T>
__device__ __forceinline__ float load_at(const void* x, long long i);
template <>
__device__ __forceinline__ float load_at<float>(const void* x, long long i) {
  return __ldg(static_cast<const float*>(x) + i);
}
template <>
__device__ __forceinline__ float load_at<bf16>(const void* x, long long i) {
  return __bfloat162float(static_cast<const bf16*>(x)[i]);
}
template <>
__device__ __forceinline__ float load_at<__half>(const void* x, long long i) {
  return __half2float(static_cast<const __half*>(x)[i]);
}

struct Shared {
  u64 red[kWarps];
  u64 hist[2048];
  u64 before;
  int bin;
  u64 table[64];
};

__device__ u64 block_sum(Shared& s, u64 v) {
  v = warp_sum64(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s.red[threadIdx.x >> 5] = v;
  __syncthreads();
  u64 t = 0;
  for (int i = 0; i < kWarps; ++i) t += s.red[i];
  return t;
}
__device__ u64 block_max(Shared& s, u64 v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s.red[threadIdx.x >> 5] = v;
  __syncthreads();
  u64 t = 0;
  for (int i = 0; i < kWarps; ++i) t = max(t, s.red[i]);
  return t;
}

// The largest key at which the running sum of `value` (keys from the largest
// down, those of at least `least`) reaches `goal`.
template <typename T, typename Value>
__device__ u64 find_cut(Shared& s, const void* x, long long at, int V, u64 least, u64 goal, Value value) {
  u64 prefix = 0;
  int shift = 64;
  u64 before = 0;
  while (shift > 0) {
    const int bits = shift >= 11 ? 11 : shift, next = shift - bits;
    for (int i = threadIdx.x; i < 2048; i += kThreads) s.hist[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < V; i += kThreads) {
      const float f = load_at<T>(x, at + i);
      const u64 k = key_of(f, i);
      if (k < least || (shift < 64 && (k >> shift) != (prefix >> shift))) continue;
      const u64 v = value(f);
      if (v) atomicAdd(&s.hist[(k >> next) & ((1 << bits) - 1)], v);
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      u64 run = before;
      int b = (1 << bits) - 1;
      while (b > 0 && run + s.hist[b] < goal) run += s.hist[b--];
      s.bin = b;
      s.before = run;
    }
    __syncthreads();
    before = s.before;
    prefix |= (u64)s.bin << next;
    shift = next;
    __syncthreads();
  }
  return prefix;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) k_sample(const __grid_constant__ SampleArgs a, const __grid_constant__ Pow2Table pow2) {
  __shared__ Shared s;
  const int row = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, V = a.V;
  const long long at = (long long)row * a.ld;
  if (tid < 64) s.table[tid] = pow2.t[tid];
  u64 best = 0;
  for (int i = tid; i < V; i += kThreads) best = max(best, key_of(load_at<T>(a.x, at + i), i));
  best = block_max(s, best);
  const float m = value_of((uint32_t)(best >> 32));
  const float temp = a.set.d_temperature ? a.set.d_temperature[row] : a.set.temperature;
  const int first = (int)(0xffffffffu - (uint32_t)best);
  if (!(fabsf(m) < INFINITY) || !(temp > 0.f)) {
    if (tid == 0) {
      a.token[row] = first;
      if (a.logprob) a.logprob[row] = fabsf(m) < INFINITY ? 0.f : NAN;
    }
    return;
  }
  const int k = a.set.d_top_k ? a.set.d_top_k[row] : a.set.top_k;
  const float tp = a.set.d_top_p ? a.set.d_top_p[row] : a.set.top_p, mp = a.set.d_min_p ? a.set.d_min_p[row] : a.set.min_p;
  const double c = fmin(1.4426950408889634 / (double)temp, 1e38);  // (finite in fp32)
  Weight w{m, (float)c, (float)(c - (double)(float)c), s.table};
  u64 cut = 0;
  if (k >= 1 && k < V) cut = find_cut<T>(s, a.x, at, V, 0, (u64)k, [](float) -> u64 { return 1; });
  if (tp < 1.f) {
    u64 sum = 0;
    for (int i = tid; i < V; i += kThreads) {
      const float f = load_at<T>(a.x, at + i);
      if (key_of(f, i) >= cut) sum += w(f);
    }
    sum = block_sum(s, sum);
    // top_p S, rounded up
    const u64 p64 = (u64)(fmax((double)tp, 0.0) * 18446744073709551616.0);
    const u64 goal = max(1ull, __umul64hi(p64, sum) + (p64 * sum != 0));
    cut = max(cut, find_cut<T>(s, a.x, at, V, cut, goal, w));
  }
  if (mp > 0.f) {
    const double b = (double)m + (double)temp * log((double)mp);
    float f = (float)b;
    if ((double)f < b) f = nextafterf(f, INFINITY);
    cut = max(cut, (u64)order_bits(f) << 32);
  }
  cut = min(cut, best);
  // the weights of each warp's share, of the warps in front, and of all
  const int per = (V + kWarps - 1) / kWarps, i0 = min(V, warp * per), i1 = min(V, i0 + per);
  u64 sum = 0;
  for (int i = i0 + lane; i < i1; i += 32) {
    const float f = load_at<T>(a.x, at + i);
    if (key_of(f, i) >= cut) sum += w(f);
  }
  sum = warp_sum64(sum);
  __syncthreads();
  if (lane == 0) s.red[warp] = sum;
  __syncthreads();
  u64 all = 0, before = 0;
  for (int i = 0; i < kWarps; ++i) {
    if (i < warp) before += s.red[i];
    all += s.red[i];
  }
  const float u = fminf(fmaxf(a.u[row], 0.f), 1.f - 5.9604644775390625e-8f);
  const u64 goal = __umul64hi((u64)((double)u * 18446744073709551616.0), all);
  if (before <= goal && goal < before + sum) {
    u64 run = before;
    for (int i = i0; i < i1; i += 32) {
      u64 v = 0;
      if (i + lane < i1) {
        const float f = load_at<T>(a.x, at + i + lane);
        if (key_of(f, i + lane) >= cut) v = w(f);
      }
      u64 inc = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const u64 t = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += t;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, run + inc > goal);
      if (hit) {
        if (lane == __ffs(hit) - 1) {
          a.token[row] = i + lane;
          if (a.logprob) a.logprob[row] = logf((float)v / (float)all);
        }
        break;
      }
      run += __shfl_sync(0xffffffffu, inc, 31);
    }
  }
}

}  // namespace

cudaError_t launch_sample(const SampleArgs& a, cudaStream_t s) {
  static const Pow2Table table = [] {
    Pow2Table t;
    for (int j = 0; j < 64; ++j) t.t[j] = (u64)llrint(exp2(44.0 - j / 64.0));
    return t;
  }();
  if (a.dtype == RL_DT_F32)
    k_sample<float><<<a.rows, kThreads, 0, s>>>(a, table);
  else if (a.dtype == RL_DT_BF16)
    k_sample<bf16><<<a.rows, kThreads, 0, s>>>(a, table);
  else
    k_sample<__half><<<a.rows, kThreads, 0, s>>>(a, table);
  return cudaGetLastError();
}

}  // namespace river

using namespace river;

extern "C" rl_status rl_sample(const void* d_logits, int32_t dtype, int32_t rows, int32_t vocab, int64_t row_stride,
                               const float* d_u, const rl_sampling* settings, int32_t* d_token, float* d_logprob,
                               int32_t* d_err, rl_stream_t stream) {
  auto bad = [](rl_status st, const char* what) {
    char msg[256];
    snprintf(msg, sizeof(msg), "rl_sample: %s", what);
    return set_error(st, msg);
  };
  if (!d_logits || !d_u || !settings || !d_token) return bad(RL_ERR_INVALID_ARG, "NULL argument");
  if (dtype != RL_DT_F32 && dtype != RL_DT_BF16 && dtype != RL_DT_F16) return bad(RL_ERR_INVALID_ARG, "unknown dtype");
  if (rows < 1 || vocab < 1 || row_stride < vocab) return bad(RL_ERR_INVALID_ARG, "rows and vocab must be >= 1, row_stride >= vocab");
  if (vocab > 1 << 19) return bad(RL_ERR_UNSUPPORTED, "vocab must be at most 2^19");
  const rl_sampling& s = *settings;
  if ((!s.d_temperature && !(s.temperature >= 0.f && s.temperature < INFINITY)) || (!s.d_top_k && s.top_k < 0) ||
      (!s.d_top_p && !(s.top_p >= 0.f && s.top_p < INFINITY)) || (!s.d_min_p && !(s.min_p >= 0.f && s.min_p < INFINITY)))
    return bad(RL_ERR_INVALID_ARG, "temperature, top_k, top_p and min_p must not be negative, nor NaN or infinite");
  if (reinterpret_cast<uintptr_t>(d_logits) % (dtype == RL_DT_F32 ? 4 : 2)) return bad(RL_ERR_INVALID_ARG, "logits off their element's alignment");
  SampleArgs a = {};
  a.x = d_logits;
  a.dtype = dtype;
  a.rows = rows;
  a.V = vocab;
  a.ld = row_stride;
  a.u = d_u;
  a.set = s;
  a.token = d_token;
  a.logprob = d_logprob;
  a.err = d_err;
  const cudaError_t e = launch_sample(a, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return set_error(RL_ERR_CUDA, cudaGetErrorString(e));
  return RL_OK;
}
