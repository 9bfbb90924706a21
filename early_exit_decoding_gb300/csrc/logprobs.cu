// Log-probabilities of given tokens, entropy and top alternatives of rows of
// logits (rl_token_logprobs).
//
// With m = max x, s = sum exp(x - m) and t = sum (x - m) exp(x - m):
//   lse = m + ln s,  entropy = ln s - t / s,  logprob_i = (x_i - m) - ln s.
// One pass over the row.  Every thread keeps its own (m, s, t): a tile of 16
// (fp32) or 32 (bf16, fp16) logits a thread raises m by the tile's maximum
// first, s' = a s and t' = a (t + (m - m') s) with a = exp(m - m'), then adds
// the tile's terms; threads, warps and the CTAs of a cluster join theirs by
// the same rule in a fixed order, so results repeat bit for bit.
//
// Top k (k <= 32): every warp keeps the candidates above its threshold in a
// list in shared memory, as 64-bit keys (ordered value, then the lower id).
// The first threshold is the k-th largest of the 32 lanes' maxima in the
// first tile (at least k logits reach it); a full list is cut to its k
// largest, the last of which is the next threshold.  A tile none of whose
// logits reaches the threshold costs one comparison a thread and one vote.
// The warps' lists are merged in order, then the CTAs'.
//
// A few rows are split over a thread-block cluster each (up to 16 CTAs); its
// CTAs exchange sums and candidates through distributed shared memory, so
// there is no workspace and no second launch.
#include <float.h>
#include <math.h>

#include <atomic>
#include <mutex>

#include "dev_common.cuh"
#include "internal.h"

namespace river {

namespace {

using namespace dev;

constexpr int kLpThreads = 512;
constexpr int kLpWarps = kLpThreads / 32;
constexpr int kLpVecs = 4;       // 16-byte loads of a thread's tile
constexpr int kLpCap = 128;      // candidates a warp's list holds
constexpr int kLpMaxSplit = 16;  // CTAs of a row's cluster
constexpr float kLog2e = 1.4426950408889634f;

// Unsigned keys that order values as documented: NaN above +infinity, -0 as
// +0; the low half orders equal values by the lower id.
__device__ __forceinline__ uint32_t order_bits(float x) {
  const uint32_t u = x != x ? 0x7fffffffu : __float_as_uint(x + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ unsigned long long order_key(float x, int id) {
  return ((unsigned long long)order_bits(x) << 32) | (0xffffffffu - (uint32_t)id);
}
__device__ __forceinline__ unsigned long long warp_max_u64(unsigned long long v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const unsigned long long w = __shfl_xor_sync(0xffffffffu, v, o);
    v = w > v ? w : v;
  }
  return v;
}
// Maximum that a NaN survives.
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <typename T>
struct Elem;
template <>
struct Elem<float> {
  static constexpr int kVec = 4;
  static constexpr uint32_t kNegInf = 0xff800000u;
  static __device__ __forceinline__ float get(const uint4& v, int e) { return __uint_as_float(u4get(v, e)); }
  static __device__ __forceinline__ float load(const float* p) { return *p; }
  static __device__ __forceinline__ void set(uint32_t (&w)[4], int e, const float* p) { w[e] = __float_as_uint(*p); }
};
template <>
struct Elem<bf16> {
  static constexpr int kVec = 8;
  static constexpr uint32_t kNegInf = 0xff80ff80u;
  static __device__ __forceinline__ float get(const uint4& v, int e) {
    const uint32_t w = u4get(v, e >> 1);
    return __uint_as_float((e & 1) ? (w & 0xffff0000u) : (w << 16));
  }
  static __device__ __forceinline__ float load(const bf16* p) { return __bfloat162float(*p); }
  static __device__ __forceinline__ void set(uint32_t (&w)[4], int e, const bf16* p) {
    const uint32_t b = *reinterpret_cast<const uint16_t*>(p);
    w[e >> 1] = (e & 1) ? (w[e >> 1] & 0xffffu) | (b << 16) : (w[e >> 1] & 0xffff0000u) | b;
  }
};
template <>
struct Elem<__half> {
  static constexpr int kVec = 8;
  static constexpr uint32_t kNegInf = 0xfc00fc00u;
  static __device__ __forceinline__ float get(const uint4& v, int e) {
    const uint32_t w = u4get(v, e >> 1);
    return __half2float(__ushort_as_half((unsigned short)((e & 1) ? w >> 16 : w & 0xffffu)));
  }
  static __device__ __forceinline__ float load(const __half* p) { return __half2float(*p); }
  static __device__ __forceinline__ void set(uint32_t (&w)[4], int e, const __half* p) {
    const uint32_t b = *reinterpret_cast<const uint16_t*>(p);
    w[e >> 1] = (e & 1) ? (w[e >> 1] & 0xffffu) | (b << 16) : (w[e >> 1] & 0xffff0000u) | b;
  }
};

// Partial sums of a part of a row: s and t relative to m.
struct Part {
  float m, s, t;
};
// The point exponentials are taken from: m, or 0 while nothing above
// -infinity has been seen (exp(-infinity - 0) = 0).
__device__ __forceinline__ float pivot(float m) { return m == -INFINITY ? 0.f : m; }
__device__ __forceinline__ void rebase(Part& p, float m_new) {
  // the clamp keeps 0 * infinity out of t (and drops what an empty part, m
  // -infinity, does not hold); a NaN passes it
  const float d = max_nan(p.m - pivot(m_new), -1e30f), a = ex2(d * kLog2e);
  p.t = a * (p.t + d * p.s);
  p.s *= a;
  p.m = m_new;
}
__device__ __forceinline__ Part join(Part x, Part y) {
  const float m = fmaxf(x.m, y.m);
  rebase(x, m);
  rebase(y, m);
  return Part{m, x.s + y.s, x.t + y.t};
}

// A warp's candidate list: `cnt` keys, of which those above `thr` matter.
struct Cand {
  unsigned long long* list;
  unsigned long long thr;
  float thr_f;
  int cnt;
};

__device__ __forceinline__ float value_of(unsigned long long key) {
  const uint32_t o = (uint32_t)(key >> 32);
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7fffffffu) : ~o);
}

// Keeps the k largest keys of the list, largest first.
__device__ __noinline__ void cut_list(Cand& c, int k, int lane) {
  __syncwarp();
  unsigned long long v[kLpCap / 32];
#pragma unroll
  for (int i = 0; i < kLpCap / 32; ++i) v[i] = lane + 32 * i < c.cnt ? c.list[lane + 32 * i] : 0ull;
  __syncwarp();
  const int n = min(k, c.cnt);
  unsigned long long last = ~0ull, mine = 0;
  for (int r = 0; r < n; ++r) {  // keys differ, so "below the last one" is the rest
    unsigned long long b = 0;
#pragma unroll
    for (int i = 0; i < kLpCap / 32; ++i) b = (v[i] < last && v[i] > b) ? v[i] : b;
    last = warp_max_u64(b);
    if (lane == r) mine = last;
  }
  if (lane < n) c.list[lane] = mine;
  c.cnt = n;
  if (n == k) {
    c.thr = last;
    c.thr_f = value_of(last);
  }
  __syncwarp();
}

template <typename T, bool kTop>
__global__ void __launch_bounds__(kLpThreads, 2) k_logprobs(LogprobArgs a, int split) {
  using E = Elem<T>;
  constexpr int VEC = E::kVec, N = kLpVecs * VEC;
  __shared__ Part s_part[kLpWarps];
  __shared__ Part s_cta;
  __shared__ unsigned long long s_list[kTop ? kLpWarps : 1][kTop ? kLpCap : 1];
  __shared__ unsigned long long s_top[kTop ? 32 : 1];
  __shared__ unsigned long long s_all[kTop ? kLpMaxSplit : 1][kTop ? 32 : 1];

  const int row = blockIdx.x / split, part = blockIdx.x % split;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const T* x = static_cast<const T*>(a.x) + (long long)row * a.ld;
  const int V = a.V, k = a.top_k;

  // The row in 16-byte vectors: vector 0 holds the first logit at element
  // `mis`; the first and last vector may reach outside the row.
  const int mis = (int)((reinterpret_cast<uintptr_t>(x) & 15) / sizeof(T));
  const T* xv = x - mis;
  const int nvec = (int)(((long long)V + mis + VEC - 1) / VEC);
  const int v0 = (int)((long long)nvec * part / split), v1 = (int)((long long)nvec * (part + 1) / split);

  auto fetch = [&](int v) -> uint4 {
    uint32_t w[4] = {E::kNegInf, E::kNegInf, E::kNegInf, E::kNegInf};
    if (v < v1) {
      const long long e0 = (long long)v * VEC - mis;
      if (e0 >= 0 && e0 + VEC <= V) return __ldcs(reinterpret_cast<const uint4*>(xv + (long long)v * VEC));
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        if (e0 + e >= 0 && e0 + e < V) E::set(w, e, x + e0 + e);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  };

  Part p{-INFINITY, 0.f, 0.f};
  Cand c{kTop ? s_list[warp] : nullptr, 0ull, -INFINITY, 0};
  bool first = true;
  uint4 nxt[kLpVecs];
#pragma unroll
  for (int j = 0; j < kLpVecs; ++j) nxt[j] = fetch(v0 + j * kLpThreads + tid);
  for (int base = v0; base < v1; base += kLpVecs * kLpThreads) {
    uint4 cur[kLpVecs];
#pragma unroll
    for (int j = 0; j < kLpVecs; ++j) cur[j] = nxt[j];
    if (base + kLpVecs * kLpThreads < v1) {
#pragma unroll
      for (int j = 0; j < kLpVecs; ++j) nxt[j] = fetch(base + (kLpVecs + j) * kLpThreads + tid);
    }
    float tm = E::get(cur[0], 0);
#pragma unroll
    for (int i = 1; i < N; ++i) tm = max_nan(tm, E::get(cur[i / VEC], i % VEC));
    const float mn = fmaxf(p.m, tm);
    if (mn > p.m) rebase(p, mn);
    const float mu = pivot(p.m);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float d = max_nan(E::get(cur[i / VEC], i % VEC) - mu, -1e30f);
      const float e = ex2(d * kLog2e);
      p.s += e;
      p.t = fmaf(d, e, p.t);
    }
    if constexpr (kTop) {
      if (first) {
        // the k-th largest of the lanes' maxima: at least k logits reach it
        first = false;
        const uint32_t o = order_bits(tm);
        int rank = 0;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const uint32_t q = __shfl_sync(0xffffffffu, o, i);
          rank += q > o || (q == o && i < lane);
        }
        const unsigned who = __ballot_sync(0xffffffffu, rank == k - 1);
        const uint32_t ok = __shfl_sync(0xffffffffu, o, __ffs(who) - 1);
        c.thr = ((unsigned long long)ok << 32) - 1;
        c.thr_f = value_of((unsigned long long)ok << 32);
      }
      if (__any_sync(0xffffffffu, !(tm < c.thr_f))) {
#pragma unroll 1
        for (int j = 0; j < kLpVecs; ++j) {
          uint4 cv = cur[0];
          if (j == 1) cv = cur[1];
          if (j == 2) cv = cur[2];
          if (j == 3) cv = cur[3];
          const long long e0 = (long long)(base + j * kLpThreads + tid) * VEC - mis;
          const bool in = base + j * kLpThreads + tid < v1;
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            const float v = E::get(cv, e);
            const unsigned long long key = order_key(v, (int)(e0 + e));
            const bool take = in && key > c.thr && e0 + e >= 0 && e0 + e < V;
            const unsigned mask = __ballot_sync(0xffffffffu, take);
            if (mask) {
              if (take) c.list[c.cnt + __popc(mask & ((1u << lane) - 1))] = key;
              c.cnt += __popc(mask);
              if (c.cnt > kLpCap - 32) cut_list(c, k, lane);
            }
          }
        }
      }
    }
  }

#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    p = join(p, Part{__shfl_xor_sync(0xffffffffu, p.m, o), __shfl_xor_sync(0xffffffffu, p.s, o),
                     __shfl_xor_sync(0xffffffffu, p.t, o)});
  if (lane == 0) s_part[warp] = p;
  if constexpr (kTop) {
    cut_list(c, k, lane);
    for (int i = c.cnt + lane; i < k; i += 32) c.list[i] = 0ull;
  }
  __syncthreads();
  // `src(i)`: list of k keys, largest first, zeros behind; the k largest of n lists in order
  auto merge = [&](auto src, int n, unsigned long long* out) {
    int at = 0;
    for (int r = 0; r < k; ++r) {
      const unsigned long long h = lane < n && at < k ? src(lane)[at] : 0ull;
      const unsigned long long b = warp_max_u64(h);
      if (lane < n && h == b && b != 0) ++at;
      if (lane == 0) out[r] = b;
    }
    __syncwarp();
  };
  if (warp == 0) {
    p = lane < kLpWarps ? s_part[lane] : Part{-INFINITY, 0.f, 0.f};
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      p = join(p, Part{__shfl_xor_sync(0xffffffffu, p.m, o), __shfl_xor_sync(0xffffffffu, p.s, o),
                       __shfl_xor_sync(0xffffffffu, p.t, o)});
    if (lane == 0) s_cta = p;
    if constexpr (kTop) merge([&](int i) { return s_list[i]; }, kLpWarps, s_top);
  }
  if (split > 1) {
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (part == 0 && warp == 0) {
      auto remote = [&](const void* q, int rank) {
        uint32_t r;
        asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(q)), "r"(rank));
        return r;
      };
      p = Part{-INFINITY, 0.f, 0.f};
      if (lane < split) {
        const uint32_t at = remote(&s_cta, lane);
        asm volatile("ld.shared::cluster.f32 %0, [%3];\nld.shared::cluster.f32 %1, [%3+4];\nld.shared::cluster.f32 %2, [%3+8];"
                     : "=f"(p.m), "=f"(p.s), "=f"(p.t)
                     : "r"(at)
                     : "memory");
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1)
        p = join(p, Part{__shfl_xor_sync(0xffffffffu, p.m, o), __shfl_xor_sync(0xffffffffu, p.s, o),
                         __shfl_xor_sync(0xffffffffu, p.t, o)});
      if constexpr (kTop) {
        for (int i = 0; i < split; ++i) {
          if (lane < k) {
            unsigned long long v;
            asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(remote(&s_top[lane], i)) : "memory");
            s_all[i][lane] = v;
          }
        }
        __syncwarp();
        merge([&](int i) { return s_all[i]; }, split, s_top);
      }
    }
    // nobody leaves while its shared memory may still be read
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (part != 0) return;
  }
  if (warp != 0) return;
  const float m = __shfl_sync(0xffffffffu, p.m, 0), s = __shfl_sync(0xffffffffu, p.s, 0), t = __shfl_sync(0xffffffffu, p.t, 0);
  // no distribution: nothing above -infinity (s 0), or a NaN or +infinity (s NaN)
  const float ln_s = s == 0.f ? NAN : logf(s);
  if (lane == 0) {
    if (a.lse) a.lse[row] = s == 0.f ? -INFINITY : m + ln_s;
    if (a.entropy) a.entropy[row] = ln_s - t / s;
  }
  for (int i = lane; i < a.n_tok; i += 32) {
    const int tok = a.tokens[(long long)row * a.n_tok + i];
    float v = NAN;
    if (tok >= 0 && tok < V)
      v = (E::load(x + tok) - m) - ln_s;
    else if (a.err)
      atomicOr(a.err, RL_DEVERR_TOKEN);
    a.logprob[(long long)row * a.n_tok + i] = v;
  }
  if constexpr (kTop) {
    if (lane < k) {
      const int id = (int)(0xffffffffu - (uint32_t)s_top[lane]);
      a.top_ids[(long long)row * k + lane] = id;
      a.top_lp[(long long)row * k + lane] = (E::load(x + id) - m) - ln_s;
    }
  }
}

// CTAs a row is split over: one while the rows fill the GPU's resident CTAs
// (two a SM); else as many as keep them busy, not below one tile each.
int pick_split(int rows, long long vecs, int sm_count) {
  int s = 1;
  while (s < kLpMaxSplit && rows * s * 2 <= 2 * sm_count && vecs > (long long)s * kLpThreads * kLpVecs) s *= 2;
  return s;
}

template <typename T, bool kTop>
cudaError_t launch(const LogprobArgs& a, cudaStream_t s) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  e = device_sm_count(dev, &sms);
  if (e != cudaSuccess) return e;
  auto kern = k_logprobs<T, kTop>;
  {
    // once per device: clusters above 8 CTAs need the opt-in
    static std::mutex mu;
    static bool done[kOpDevices] = {};
    std::lock_guard<std::mutex> lock(mu);
    if (!done[dev]) {
      e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
      if (e != cudaSuccess) return e;
      done[dev] = true;
    }
  }
  const int split = pick_split(a.rows, ((long long)a.V + Elem<T>::kVec - 1) / Elem<T>::kVec, sms);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.rows * split);
  cfg.blockDim = dim3(kLpThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = split;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, a, split);
}

}  // namespace

cudaError_t device_sm_count(int dev, int* out) {
  static std::atomic<int> count[kOpDevices];
  if (dev < 0 || dev >= kOpDevices) return cudaErrorInvalidDevice;
  int n = count[dev].load();
  if (n == 0) {
    const cudaError_t e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    count[dev].store(n);
  }
  *out = n;
  return cudaSuccess;
}

cudaError_t launch_logprobs(const LogprobArgs& a, cudaStream_t s) {
  const bool top = a.top_k > 0;
  if (a.dtype == RL_DT_F32) return top ? launch<float, true>(a, s) : launch<float, false>(a, s);
  if (a.dtype == RL_DT_BF16) return top ? launch<bf16, true>(a, s) : launch<bf16, false>(a, s);
  return top ? launch<__half, true>(a, s) : launch<__half, false>(a, s);
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
