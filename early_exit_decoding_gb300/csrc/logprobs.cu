// Log-probabilities of given tokens, entropy and top alternatives of rows of
// logits (rl_token_logprobs).
//
// With m = max x, s = sum exp(x - m) and t = sum (x - m) exp(x - m):
//   lse = m + ln s,  entropy = ln s - t / s,  logprob_i = (x_i - m) - ln s.
// One pass over the row.  Every warp has its own ring of 2 KB tiles filled by
// bulk copies (192 KB in flight a SM without a register held for them; plain
// loads prefetched into registers spilled and gave 5.3 TB/s).  Every thread
// keeps its own (m, s, t): a tile of 16 (fp32) or 32 (bf16, fp16) logits a
// thread raises m to the tile's maximum first, s' = a s and
// t' = a (t + (m - m') s) with a = exp(m - m'), then adds the tile's terms;
// threads, warps and the CTAs of a cluster join theirs by
// the same rule in a fixed order, so results repeat bit for bit.
//
// Top k (k <= 32): every warp keeps the candidates above its threshold in a
// list in shared memory, as 64-bit keys (ordered value, then the lower id).
// The first threshold is the k-th largest of the four largest thread maxima of
// each of the 8 warps' first tiles (at least k logits reach it: for k = 20
// about 1 % of random logits do); a full list is cut to its k
// largest, the last of which is the next threshold.  A tile none of whose
// logits reaches the threshold costs one comparison a thread and one vote.
// The warps' lists are merged in order, then the CTAs'.
//
// What bounds it: HBM at many rows (4096 rows of 128,256 fp32 logits: 302 us,
// 6.95 TB/s, 1.02 of a measured copy); at few rows the chain of a launch, the
// copies' first arrival and the joins of warps and CTAs (one row 7.6 us, of
// 0.5 MB), with top k above all the candidates' selection (64 rows: 10.1 us
// without, 19.7 with 20 alternatives).  16-bit rows bring twice the logits a
// byte and every logit is unpacked, so instructions bind them before HBM (777
// odd rows of 50,257 bf16 logits: 33 us, 17 of them issue slots, 2.4 TB/s).
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

constexpr int kLpThreads = 256;
constexpr int kLpWarps = kLpThreads / 32;
constexpr int kLpResident = 4;   // CTAs a SM holds
constexpr int kLpVecs = 4;       // 16-byte vectors of a thread's tile
constexpr int kLpTile = 32 * kLpVecs;           // vectors of a warp's tile
constexpr int kLpStages = 3;     // tiles of a warp's ring
constexpr int kLpRing = kLpWarps * kLpStages * kLpTile * 16;
constexpr int kLpCap = 96;       // candidates a warp's list holds (4 CTAs' shared memory fits an SM)
constexpr int kLpMaxSplit = 16;  // CTAs of a row's cluster
constexpr unsigned long long kLpWaitNs = 2000000000ull;  // a wait gives up after two seconds
constexpr float kLog2e = 1.4426950408889634f;
static_assert(kLpWarps == 8 && kLpVecs == 4, "the first threshold takes four values of each of 8 warps");

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
  const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(v >> 32));
  const uint32_t lo = __reduce_max_sync(0xffffffffu, (uint32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
  return ((unsigned long long)hi << 32) | lo;
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
  static constexpr uint32_t kNegInf = 0xff800000u;  // -infinity in every element
  static __device__ __forceinline__ float get(const uint4& v, int e) { return __uint_as_float(u4get(v, e)); }
  static __device__ __forceinline__ float largest(const uint4& v) {
    return max_nan(max_nan(get(v, 0), get(v, 1)), max_nan(get(v, 2), get(v, 3)));
  }
  static __device__ __forceinline__ float load(const float* p) { return *p; }
};
template <>
struct Elem<bf16> {
  static constexpr int kVec = 8;
  static constexpr uint32_t kNegInf = 0xff80ff80u;
  static __device__ __forceinline__ float get(const uint4& v, int e) {
    const uint32_t w = u4get(v, e >> 1);
    return __uint_as_float((e & 1) ? (w & 0xffff0000u) : (w << 16));
  }
  static __device__ __forceinline__ float largest(const uint4& v) {  // (pairs at a time; exact)
    uint32_t m, n;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(v.x), "r"(v.y));
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(n) : "r"(v.z), "r"(v.w));
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(m), "r"(n));
    return max_nan(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
  }
  static __device__ __forceinline__ float load(const bf16* p) { return __bfloat162float(*p); }
};
template <>
struct Elem<__half> {
  static constexpr int kVec = 8;
  static constexpr uint32_t kNegInf = 0xfc00fc00u;
  static __device__ __forceinline__ float get(const uint4& v, int e) {
    const uint32_t w = u4get(v, e >> 1);
    return __half2float(__ushort_as_half((unsigned short)((e & 1) ? w >> 16 : w & 0xffffu)));
  }
  static __device__ __forceinline__ float largest(const uint4& v) {
    uint32_t m, n;
    asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(m) : "r"(v.x), "r"(v.y));
    asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(n) : "r"(v.z), "r"(v.w));
    asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(m) : "r"(m), "r"(n));
    return max_nan(get(make_uint4(m, 0, 0, 0), 0), get(make_uint4(m, 0, 0, 0), 1));
  }
  static __device__ __forceinline__ float load(const __half* p) { return __half2float(*p); }
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

__device__ __forceinline__ float value_of(unsigned long long key) {
  const uint32_t o = (uint32_t)(key >> 32);
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7fffffffu) : ~o);
}

// Keeps the k largest of the list's cnt keys, largest first; returns how many.
__device__ __noinline__ int cut_list(unsigned long long* list, int cnt, int k, int lane) {
  __syncwarp();
  unsigned long long v[kLpCap / 32];
#pragma unroll
  for (int i = 0; i < kLpCap / 32; ++i) v[i] = lane + 32 * i < cnt ? list[lane + 32 * i] : 0ull;
  __syncwarp();
  const int n = min(k, cnt);
  unsigned long long last = ~0ull, mine = 0;
  for (int r = 0; r < n; ++r) {  // keys differ, so "below the last one" is the rest
    unsigned long long b = 0;
#pragma unroll
    for (int i = 0; i < kLpCap / 32; ++i) b = (v[i] < last && v[i] > b) ? v[i] : b;
    last = warp_max_u64(b);
    if (lane == r) mine = last;
  }
  if (lane < n) list[lane] = mine;
  __syncwarp();
  return n;
}

// The k-th largest of the lanes' values (0: none).
__device__ __forceinline__ uint32_t kth_of_lanes(uint32_t v, int k, int lane) {
  int rank = 0;
#pragma unroll 8
  for (int i = 0; i < 32; ++i) {
    const uint32_t q = __shfl_sync(0xffffffffu, v, i);
    rank += q > v || (q == v && i < lane);
  }
  const unsigned who = __ballot_sync(0xffffffffu, rank == k - 1);
  return __shfl_sync(0xffffffffu, v, __ffs(who) - 1);
}

// The lanes' keys that reach `least` in their value join sel (counted in *n,
// beyond kLpSel counted only).
constexpr int kLpSel = 64;
__device__ __forceinline__ void select(unsigned long long key, uint32_t least, unsigned long long* sel, int* n, int lane) {
  const bool take = key != 0 && (uint32_t)(key >> 32) >= least;
  const unsigned mask = __ballot_sync(0xffffffffu, take);
  if (!mask) return;
  int at = 0;
  if (lane == __ffs(mask) - 1) at = atomicAdd(n, __popc(mask));
  at = __shfl_sync(0xffffffffu, at, __ffs(mask) - 1) + __popc(mask & ((1u << lane) - 1));
  if (take && at < kLpSel) sel[at] = key;
}
// One warp: the k largest of sel's n <= kLpSel keys in order, zeros behind
// (a key's place is the number of larger ones: the order they came in is immaterial).
__device__ __forceinline__ void rank_sel(const unsigned long long* sel, int n, int k, unsigned long long* out, int lane) {
  const unsigned long long a = lane < n ? sel[lane] : 0ull, b = lane + 32 < n ? sel[lane + 32] : 0ull;
  int ra = 0, rb = 0;
#pragma unroll 4
  for (int i = 0; i < n; ++i) {
    const unsigned long long x = sel[i];
    ra += x > a;
    rb += x > b;
  }
  if (lane >= n && lane < k) out[lane] = 0ull;
  if (a != 0 && ra < k) out[ra] = a;
  if (b != 0 && rb < k) out[rb] = b;
  __syncwarp();
}

// Two fp32 operations an instruction.
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  unsigned long long d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(d)
      : "l"(*reinterpret_cast<unsigned long long*>(&a)), "l"(*reinterpret_cast<unsigned long long*>(&b)));
  return *reinterpret_cast<float2*>(&d);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  unsigned long long d;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(d)
      : "l"(*reinterpret_cast<unsigned long long*>(&a)), "l"(*reinterpret_cast<unsigned long long*>(&b)));
  return *reinterpret_cast<float2*>(&d);
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  unsigned long long d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(d)
      : "l"(*reinterpret_cast<unsigned long long*>(&a)), "l"(*reinterpret_cast<unsigned long long*>(&b)),
        "l"(*reinterpret_cast<unsigned long long*>(&c)));
  return *reinterpret_cast<float2*>(&d);
}

// Adds one logit to a part whose m is already at least as large.
__device__ __forceinline__ void add(Part& p, float x, float mu) {
  const float d = max_nan(x - mu, -1e30f), e = ex2(d * kLog2e);
  p.s += e;
  p.t = fmaf(d, e, p.t);
}

template <typename T, bool kTop>
__global__ void __launch_bounds__(kLpThreads, kLpResident) k_logprobs(const __grid_constant__ LogprobArgs a, int log_split) {
  using E = Elem<T>;
  constexpr int VEC = E::kVec;
  extern __shared__ __align__(16) unsigned char ring_all[];
  __shared__ __align__(8) uint64_t full[kLpWarps][kLpStages];
  __shared__ Part s_part[kLpWarps];
  __shared__ Part s_cta;
  __shared__ unsigned long long s_list[kTop ? kLpWarps : 1][kTop ? kLpCap : 1];
  __shared__ uint32_t s_w[32];  // four large values of each warp
  __shared__ unsigned long long s_sel[kTop ? kLpSel : 1];
  __shared__ int s_n;
  __shared__ unsigned long long s_top[kTop ? 32 : 1];

  const int split = 1 << log_split, row = blockIdx.x >> log_split, part = blockIdx.x & (split - 1);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const T* x = static_cast<const T*>(a.x) + (long long)row * a.ld;
  const int V = a.V, k = a.top_k;

  // The row's whole 16-byte vectors [0, nvec) start `head` logits in; this
  // CTA's part of them is [v0, v1), dealt out to its warps in tiles of 2 KB.
  // The logits in front (part 0) and behind (last part) are `edge`, one a lane
  // of warp 0.
  const int head = min(V, (int)((16 - (reinterpret_cast<uintptr_t>(x) & 15)) % 16 / sizeof(T)));
  const int nvec = (V - head) / VEC;
  const int v0 = (int)((long long)nvec * part >> log_split), v1 = (int)((long long)nvec * (part + 1) >> log_split);
  const T* xv = x + head;
  const int ntile = (v1 - v0 + kLpTile - 1) / kLpTile;
  unsigned char* ring = ring_all + warp * kLpStages * kLpTile * 16;
  auto issue = [&](int i, int st) {  // tile i of the part into stage st
    const int at = v0 + i * kLpTile, n = min(kLpTile, v1 - at);
    mbar_expect_tx(&full[warp][st], n * 16);
    bulk_g2s(ring + st * kLpTile * 16, xv + (long long)at * VEC, n * 16, &full[warp][st]);
  };
  if (tid == 0) s_n = 0;
  if (lane == 0) {
    for (int i = 0; i < kLpStages; ++i) mbar_init(&full[warp][i], 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    for (int i = 0; i < kLpStages; ++i)
      if (warp + i * kLpWarps < ntile) issue(warp + i * kLpWarps, i);
  }
  // the given tokens' logits, one a thread (part 0; n_tok <= 256)
  float tokv = NAN;
  const long long orow = row + a.row0;  // where the row's outputs go
  const int tpos = a.T > 0 ? (int)(orow % a.T) : 0;
  const int n_tok = a.T > 0 ? (tpos < a.T - 1) : a.n_tok;
  const long long tok_at = a.T > 0 ? orow + 1 : orow * a.n_tok;
  if (part == 0 && tid < n_tok) {
    const int tok = a.tokens[tok_at + tid];
    if (tok >= 0 && tok < V)
      tokv = E::load(x + tok);
    else if (a.err)
      atomicOr(a.err, RL_DEVERR_TOKEN);
  }
  Part p{-INFINITY, 0.f, 0.f};
  int edge = -1;  // id of this lane's edge logit
  float edge_v = -INFINITY;
  if (warp == 0) {
    const int rest = V - head - nvec * VEC;
    if (part == 0 && lane < head) edge = lane;
    if (part == split - 1 && lane >= 16 && lane - 16 < rest) edge = V - rest + (lane - 16);
    if (edge >= 0) {
      edge_v = E::load(x + edge);
      p.m = fmaxf(p.m, edge_v);
      add(p, edge_v, pivot(p.m));
    }
  }
  __syncwarp();

  bool ok = true;
  auto wait = [&](int st, int ph) {
    const bool got = mbar_wait_lazy(&full[warp][st], ph, kLpWaitNs);
    if (!__all_sync(0xffffffffu, got) && ok) {
      ok = false;
      if (lane == 0 && a.err) atomicOr(a.err, RL_DEVERR_TIMEOUT);
    }
  };
  auto vec = [&](int i, int st, int j) {  // this lane's vector j of tile i
    return v0 + i * kLpTile + j * 32 + lane < v1
               ? *reinterpret_cast<const uint4*>(ring + (st * kLpTile + j * 32 + lane) * 16)
               : make_uint4(E::kNegInf, E::kNegInf, E::kNegInf, E::kNegInf);
  };
  auto vec_max = [&](const uint4& v) { return E::largest(v); };

  // This warp's candidates: `cnt` keys above `thr` (thr_f: its value).
  unsigned long long* const list = s_list[kTop ? warp : 0];
  unsigned long long thr = 0;
  float thr_f = -INFINITY;
  int cnt = 0;
  auto push = [&](unsigned long long key, bool may) {
    const bool take = may && key > thr;
    const unsigned mask = __ballot_sync(0xffffffffu, take);
    if (take) list[cnt + __popc(mask & ((1u << lane) - 1))] = key;
    cnt += __popc(mask);
    if (cnt > kLpCap - 32) {
      cnt = cut_list(list, cnt, k, lane);  // (more than k were there)
      thr = list[k - 1];
      thr_f = value_of(thr);
    }
  };
  // The four largest of the lanes' values to s_w.
  auto publish4 = [&](uint32_t v) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w = __reduce_max_sync(0xffffffffu, v);
      if (lane == __ffs(__ballot_sync(0xffffffffu, v == w)) - 1) {
        s_w[4 * warp + i] = w;
        v = 0;
      }
    }
  };
  if constexpr (kTop) {
    uint32_t o = 0;
    if (warp < ntile) {
      wait(0, 0);
      o = order_bits(max_nan(max_nan(vec_max(vec(warp, 0, 0)), vec_max(vec(warp, 0, 1))),
                             max_nan(vec_max(vec(warp, 0, 2)), vec_max(vec(warp, 0, 3)))));
    }
    publish4(o);
    __syncthreads();
    const uint32_t kth = kth_of_lanes(s_w[lane], k, lane);
    if (kth) {
      thr = ((unsigned long long)kth << 32) - 1;
      thr_f = value_of((unsigned long long)kth << 32);
    }
    if (warp == 0) push(order_key(edge_v, edge), edge >= 0);
  }

  if constexpr (!kTop) {
    // a common start keeps the warps' neighbouring tiles together in time
    // (4096 rows of 128,256 fp32 logits: 392 -> 330 us)
    if (warp < ntile) wait(0, 0);
    __syncthreads();
  }
  // After a wait that gave up nothing is copied or computed any more; the
  // copies already in flight are still waited for (`stop`).
  int st = 0, ph = 0, stop = ok ? ntile : min(ntile, warp + kLpStages * kLpWarps);
  for (int i = warp; i < stop; i += kLpWarps) {
    const bool was = ok;
    wait(st, ph);
    if (was && !ok) stop = min(ntile, i + kLpStages * kLpWarps);
    if (ok) {
      uint4 cur[kLpVecs];
      float vm[kLpVecs];  // largest of each vector
#pragma unroll
      for (int j = 0; j < kLpVecs; ++j) cur[j] = vec(i, st, j);
#pragma unroll
      for (int j = 0; j < kLpVecs; ++j) vm[j] = vec_max(cur[j]);
      const float tm = max_nan(max_nan(vm[0], vm[1]), max_nan(vm[2], vm[3]));
      const float mn = fmaxf(p.m, tm);
      if (mn > p.m) rebase(p, mn);
      const float2 mu = make_float2(-pivot(p.m), -pivot(p.m)), l2e = make_float2(kLog2e, kLog2e);
      float2 s2 = make_float2(p.s, 0.f), t2 = make_float2(p.t, 0.f);
#pragma unroll
      for (int j = 0; j < kLpVecs; ++j)
#pragma unroll
        for (int e = 0; e < VEC; e += 2) {  // as add(), two logits at a time
          float2 d = add2(make_float2(E::get(cur[j], e), E::get(cur[j], e + 1)), mu);
          d = make_float2(max_nan(d.x, -1e30f), max_nan(d.y, -1e30f));
          float2 x = mul2(d, l2e);
          x = make_float2(ex2(x.x), ex2(x.y));
          s2 = add2(s2, x);
          t2 = fma2(d, x, t2);
        }
      p.s = s2.x + s2.y;
      p.t = t2.x + t2.y;
      if constexpr (kTop) {
        if (__any_sync(0xffffffffu, !(tm < thr_f))) {
#pragma unroll
          for (int j = 0; j < kLpVecs; ++j) {
            const int at = v0 + i * kLpTile + j * 32 + lane;
            uint32_t hits = 0;  // elements of the vector that may be candidates
            if (at < v1 && !(vm[j] < thr_f)) {
#pragma unroll
              for (int e = 0; e < VEC; ++e) hits |= !(E::get(cur[j], e) < thr_f) ? 1u << e : 0u;
            }
            while (__any_sync(0xffffffffu, hits != 0)) {
              const int e = hits ? __ffs(hits) - 1 : 0;
              const float v = E::load(reinterpret_cast<const T*>(ring + (st * kLpTile + j * 32 + lane) * 16) + e);
              push(order_key(v, head + at * VEC + e), hits != 0);
              hits &= hits - 1;
            }
          }
        }
      }
    }
    __syncwarp();
    if (ok && lane == 0 && i + kLpStages * kLpWarps < ntile) issue(i + kLpStages * kLpWarps, st);
    if (++st == kLpStages) {
      st = 0;
      ph ^= 1;
    }
  }
  if (!ok) p.s = NAN;  // a copy did not arrive (reported): no result

#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    p = join(p, Part{__shfl_xor_sync(0xffffffffu, p.m, o), __shfl_xor_sync(0xffffffffu, p.s, o),
                     __shfl_xor_sync(0xffffffffu, p.t, o)});
  if (lane == 0) s_part[warp] = p;
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
  // The lists' k largest: those that reach the k-th largest of four candidates
  // of each warp (k at least do; seldom many more) are ranked by one warp.
  if constexpr (kTop) {
    __syncwarp();
    unsigned long long v[kLpCap / 32];
    uint32_t o = 0;
#pragma unroll
    for (int q = 0; q < kLpCap / 32; ++q) {
      v[q] = lane + 32 * q < cnt ? list[lane + 32 * q] : 0ull;
      o = max(o, (uint32_t)(v[q] >> 32));
    }
    __syncthreads();  // (every warp has read the first threshold's values)
    publish4(o);
    __syncthreads();
    const uint32_t least = kth_of_lanes(s_w[lane], k, lane);
#pragma unroll
    for (int q = 0; q < kLpCap / 32; ++q)
      if (32 * q < cnt) select(v[q], least, s_sel, &s_n, lane);
    __syncthreads();
    if (s_n > kLpSel) {
      cnt = cut_list(list, cnt, k, lane);
      for (int q = cnt + lane; q < k; q += 32) list[q] = 0ull;
    }
  }
  __syncthreads();
  if (warp == 0) {
    p = lane < kLpWarps ? s_part[lane] : Part{-INFINITY, 0.f, 0.f};
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      p = join(p, Part{__shfl_xor_sync(0xffffffffu, p.m, o), __shfl_xor_sync(0xffffffffu, p.s, o),
                       __shfl_xor_sync(0xffffffffu, p.t, o)});
    if (lane == 0) s_cta = p;
    if constexpr (kTop) {
      if (s_n <= kLpSel)
        rank_sel(s_sel, s_n, k, s_top, lane);
      else
        merge([&](int i) { return s_list[i]; }, kLpWarps, s_top);
    }
  }
  __shared__ float s_res[2];
  if (split > 1) {
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (part == 0) {
      auto remote = [&](const void* q, int rank) {
        uint32_t r;
        asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(q)), "r"(rank));
        return r;
      };
      if (warp == 0) {
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
      }
      if constexpr (kTop) {
        // the CTAs' lists: one key a thread (two at most), then as the warps' above
        auto s_all = &s_list[0][0];  // (the warps' lists are done with)
        static_assert(kLpMaxSplit * 32 <= kLpWarps * kLpCap && kLpMaxSplit * 32 <= 2 * kLpThreads, "the CTAs' lists must fit");
        unsigned long long v[2] = {0ull, 0ull};
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int at = tid + q * kLpThreads;
          if (at < split * k)
            asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v[q]) : "r"(remote(&s_top[at % k], at / k)) : "memory");
        }
        __syncthreads();  // (warp 0 has ranked the CTA's own: s_sel, s_n and the lists are free)
#pragma unroll
        for (int q = 0; q < 2; ++q)
          if (tid + q * kLpThreads < split * k) s_all[tid + q * kLpThreads] = v[q];
        if (tid == 0) s_n = 0;
        __syncthreads();
        const int each = 32 >> log_split;  // of each of the CTAs' lists
        const int li = lane >> (5 - log_split), le = lane & (each - 1);
        const uint32_t least = kth_of_lanes(le < k ? (uint32_t)(s_all[li * k + le] >> 32) : 0u, k, lane);
#pragma unroll
        for (int q = 0; q < 2; ++q)
          if (q * kLpThreads + warp * 32 < split * k) select(v[q], least, s_sel, &s_n, lane);
        __syncthreads();
        if (warp == 0) {
          if (s_n <= kLpSel)
            rank_sel(s_sel, s_n, k, s_top, lane);
          else
            merge([&](int i) { return s_all + i * k; }, split, s_top);
        }
      }
    }
    // nobody leaves while its shared memory may still be read
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (part != 0) return;
  }
  if (warp == 0) {
    const float m = __shfl_sync(0xffffffffu, p.m, 0), s = __shfl_sync(0xffffffffu, p.s, 0);
    // no distribution: nothing above -infinity (s 0), or a NaN or +infinity (s NaN)
    const float ln_s = s == 0.f ? NAN : logf(s);
    if (lane == 0) {
      s_res[0] = m;
      s_res[1] = ln_s;
      if (a.lse) a.lse[orow] = s == 0.f ? -INFINITY : m + ln_s;
      if (a.entropy) a.entropy[orow] = ln_s - p.t / s;
      if (a.T > 0 && tpos == 0) a.logprob[orow] = 0.f;
    }
    if constexpr (kTop) {
      if (lane < k) {
        const unsigned long long key = s_top[lane];
        a.top_ids[orow * k + lane] = (int)(0xffffffffu - (uint32_t)key);
        a.top_lp[orow * k + lane] = (value_of(key) - m) - ln_s;
      }
    }
  }
  if (n_tok > 0) {
    __syncthreads();
    if (tid < n_tok) a.logprob[tok_at + tid] = (tokv - s_res[0]) - s_res[1];
  }
}

// CTAs a row is split over: as many as give every SM two (a cluster's start and
// join cost about 3 us: 16 rows of 128,256 fp32 logits take 16.9 us in one part,
// 7.2 in 4, 5.7 in 8, 5.9 in 16; 64 rows 17.5, 10.1, 11.4, 14.0; 256 rows 24.0
// in one, 41.8 in 2), not below one tile a warp.
// A power of two; returns its logarithm.
int pick_split(int rows, long long vecs, int sm_count) {
  int l = 0;
  while ((1 << l) < kLpMaxSplit && ((long long)rows << l) <= sm_count && vecs > (long long)kLpWarps * kLpTile << l) ++l;
  return l;
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
      e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kLpRing);
      if (e == cudaSuccess) e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
      if (e != cudaSuccess) return e;
      done[dev] = true;
    }
  }
  const int log_split = pick_split(a.rows, ((long long)a.V + Elem<T>::kVec - 1) / Elem<T>::kVec, sms);
  const int split = 1 << log_split;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.rows * split);
  cfg.blockDim = dim3(kLpThreads);
  cfg.dynamicSmemBytes = kLpRing;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = split;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, a, log_split);
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
