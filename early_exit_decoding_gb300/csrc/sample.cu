// Sampling from rows of logits with temperature, top-k, top-p and min-p, by a
// given random number (rl_sample).
//
// The ids ordered by (logit, lower id) are kept up to some last one, so what the
// three filters keep is a key: ids whose 64-bit key (ordered logit, then the
// lower id) is at least `cut`.  top-k's cut is the k-th largest key, top-p's the
// key at which the weights' running sum reaches top_p of their total; min-p's is
// a logit.  The token is then found among the ids of at least `cut` by running
// sums in the order of ids.
//
// A weight is a 64-bit whole number, exp((x - max) / T) 2^44 rounded: sums are
// exact whatever their order, and with exponentials good to 2^-35 of themselves
// (sample_weight.h; measured 2^-36.2) a token differs from that of exact weights
// only where u is that near a border (fp32 sums: 1 in 50 rows of 128,256 logits
// with a long tail).
//
// A cluster of CTAs takes a row, each a part whose warps have contiguous
// segments, and reads it from HBM once and then from L2 (held in shared memory
// no more than half of 64 rows of 128,256 fit the SMs at once: 91 us).  A cut is
// found a digit of 9 bits at a time from a histogram of the ids that agree in
// the digits before (counts, or weights in three limbs of 16 bits, whose sums
// over a part of at most 65,536 ids stay in 32); the digits are those of -log2 of
// the weight first, in fixed point (even bins where weights matter), then of the
// logit's bits and of the id, until no more than kList ids are left, which are
// ordered one against another.  A small top-k needs no histogram of the row: bins
// of the threads' largest logits give a bound that at least k ids reach and few
// others, and one CTA finishes with those alone.
//
// What bounds it: the chain of a digit (histogram, barrier, the groups' and the
// bins' sums from the other parts: three block and one cluster barrier), and
// instructions, some 77 a logit where weights are summed (the exponential's 47,
// the histogram's 20).  64 rows of 128,256 fp32 logits cut at 0.9 of their mass:
// 74 us, 45 M warp instructions (the row's first reading 7 us, the histogram 16,
// the next digit 11, the id 5, the rest between them); 500 rows of 50,257 bf16
// logits, each with settings of its own: 104 us, 64 M; one row with top-k 50 and
// top-p 0.95: 14 us.
#include <float.h>
#include <math.h>
#include <stdio.h>

#include <mutex>
#include <type_traits>

#include "dev_common.cuh"
#include "internal.h"
#include "sample_weight.h"

namespace river {

struct SampleArgs {
  const void* x;
  int dtype, rows, V;
  long long ld;
  const float* u;
  rl_sampling set;
  int* token;
  float* logprob;
};

namespace {

using namespace dev;
using u64 = unsigned long long;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxSplit = 16;    // CTAs of a row's cluster
constexpr int kBins = kThreads;  // of a digit (9 bits), one a thread
constexpr int kList = 128;       // ids that are ordered one against another
constexpr int kFew = 96;         // top-k that needs no histogram of the row
constexpr int kGather = 1024;    // a part's ids of a digit's bin that are brought together before the next digit
constexpr int kMostIds = 65536;  // of a part
constexpr int kOrder = 2048;     // rows that are put in order of their cost

__device__ __forceinline__ uint32_t order_bits(float x) {
  const uint32_t u = x != x ? 0x7fffffffu : __float_as_uint(x + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t o) {
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7fffffffu) : ~o);
}
__device__ __forceinline__ u64 key_of(float x, int id) { return ((u64)order_bits(x) << 32) | (0xffffffffu - (uint32_t)id); }

struct Pow2Table {
  u64 t[64];  // weight::entry
};

// A logit's weight (sample_weight.h), with the row's largest logit and rate.
struct Weight {
  float m, ch, cl;
  uint32_t table;  // Pow2Table in shared memory
  __device__ __forceinline__ u64 operator()(float x) const {
    return weight::of(x, m, weight::Rate{ch, cl}, [&](uint32_t j) {
      u64 t;
      asm("ld.shared.u64 %0, [%1];" : "=l"(t) : "r"(table + j * 8));
      return t;
    });
  }
};

__device__ __forceinline__ u64 warp_sum64(u64 v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ u64 warp_scan64(u64 v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 t = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += t;
  }
  return v;
}

__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t remote(const void* p, int rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
  return r;
}
__device__ __forceinline__ u64 remote64(const u64* p, int rank) {
  u64 v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(remote(p, rank)) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t remote32(const uint32_t* p, int rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(remote(p, rank)) : "memory");
  return v;
}

struct List {
  uint32_t n;
  u64 key[kList];
};
struct Shared {
  u64 table[64];
  uint32_t hist[2][4][kBins];  // by a digit's parity: counts, weights' limbs
  List list[2];                // this part's ids that are ordered one against another: for top-k, for top-p
  u64 key[kList], wt[kList];   // the cluster's, and their weights
  int n_key;
  uint32_t n_few;
  u64 few[kGather];
  u64 red[kWarps], sums[kWarps];
  u64 best, mass;           // this part's largest key, and weights kept
  u64 group[2][kWarps];     // by a digit's parity: this part's sums of 32 bins
  u64 of_bin[kMaxSplit][32];       // the parts' sums and ids in the bins of a group
  uint32_t in_bin[kMaxSplit][32];
  u64 before;               // in front of the digit's bin
  float lo, hi;             // the logits whose digits so far are the cut's
  u64 cut;
  uint32_t count, own;      // ids of the bin, and this part's
  int bin, row;
  float ch, cl, least;      // log2(e) / T in two parts; min-p's logit
  double span;              // T ln min_p
};

// An id's place in the order as digits of 9 bits from the largest down: of q, the
// complement of -log2 of its weight in fixed point (levels 0-3), of o, the ordered
// logit (4-7), and of i, the complement of the id (8-10).
struct Place {
  uint32_t q, o, i;
};
constexpr int kLevels = 11;
__device__ __forceinline__ int shift_of(int level) {  // of the field: 23, 14, 5, 0 (20 bits of ~id: 11, 2, 0)
  const int l = level & 3;
  return level < 8 ? (l == 0 ? 23 : l == 1 ? 14 : l == 2 ? 5 : 0) : (l == 0 ? 11 : l == 1 ? 2 : 0);
}
__device__ __forceinline__ int bits_of(int level) { return level < 8 ? ((level & 3) == 3 ? 5 : 9) : level == 10 ? 2 : 9; }

// Whether sums of `front` and then `more` pass from below a goal (of 1 at least) to it.
__device__ __forceinline__ bool reaches(u64 goal, u64 front, u64 more) { return goal - 1 - front < more; }

// A key that parts ids: those of a larger logit, or of its own and no higher id.
struct Cut {
  float v;
  uint32_t id;
  __device__ __forceinline__ bool takes(float x, int i) const { return x > v || (x == v && (uint32_t)i <= id); }
};
__device__ __forceinline__ Cut cut_of(u64 key) {  // 0: takes every id
  return Cut{key ? value_of((uint32_t)(key >> 32)) : -INFINITY, 0xffffffffu - (uint32_t)key};
}

// 16 bytes of logits.
template <typename T>
struct Vec {
  static constexpr int kN = 16 / sizeof(T);
  float v[kN];
  __device__ __forceinline__ explicit Vec(const uint4& x) {
#pragma unroll
    for (int e = 0; e < kN; ++e) {
      if constexpr (sizeof(T) == 4) {
        v[e] = __uint_as_float(u4get(x, e));
      } else {
        const uint32_t h = u4get(x, e >> 1);
        if constexpr (std::is_same<T, bf16>::value)
          v[e] = __uint_as_float(e & 1 ? h & 0xffff0000u : h << 16);
        else
          v[e] = __half2float(__ushort_as_half((unsigned short)(e & 1 ? h >> 16 : h & 0xffffu)));
      }
    }
  }
};

template <typename T>
struct Row {
  static constexpr int VE = Vec<T>::kN;
  Shared& s;
  const T* x;          // this part's logits from the 16-byte boundary in front of them on
  int off, end;        // where they start and end (elements)
  int first, id0, id1;  // id of the first vector's first element; this part's ids
  int i0, i1;          // this warp's segment (vectors)
  int split, tid, lane, warp;
  float m;
  Weight w;

  __device__ __forceinline__ int id(int vec, int e) const { return first + vec * VE + e; }
  // Vector i; what is not of this part is -infinity (and not read).
  __device__ __forceinline__ uint4 load(int i) const {
    if (i * VE >= off && (i + 1) * VE <= end) return __ldg(reinterpret_cast<const uint4*>(x) + i);
    return edge(i);
  }
  __device__ __noinline__ uint4 edge(int i) const {
    constexpr uint32_t none = sizeof(T) == 4 ? 0xff800000u : std::is_same<T, bf16>::value ? 0xff80u : 0xfc00u;
    uint32_t w[4] = {};
#pragma unroll
    for (int k = 0; k < VE; ++k) {
      const int at = i * VE + k;
      uint32_t v = none;
      if (at >= off && at < end) v = sizeof(T) == 4 ? reinterpret_cast<const uint32_t*>(x)[at] : reinterpret_cast<const uint16_t*>(x)[at];
      w[k * 4 / VE] |= v << (sizeof(T) == 4 ? 0 : k % 2 * 16);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  // f(logit, id) of every element of vectors b .. e - 1, the lanes' in turn, the
  // next U vectors on their way meanwhile
  template <int U, typename F>
  __device__ __forceinline__ void each(int b, int e, F f) const {
    uint4 next[U];
    const uint32_t none = sizeof(T) == 4 ? 0xff800000u : std::is_same<T, bf16>::value ? 0xff80ff80u : 0xfc00fc00u;
#pragma unroll
    for (int q = 0; q < U; ++q) next[q] = b + lane + 32 * q < e ? load(b + lane + 32 * q) : make_uint4(none, none, none, none);
    for (int i = b + lane; i < e; i += 32 * U) {
#pragma unroll
      for (int q = 0; q < U; ++q) {
        const Vec<T> v(next[q]);
        const int j = i + 32 * q;
        if (j + 32 * U < e) next[q] = load(j + 32 * U);
        if (j < e) {
#pragma unroll
          for (int k = 0; k < VE; ++k) f(v.v[k], id(j, k));
        }
      }
    }
  }
  __device__ __forceinline__ u64 mass(int b, int e, const Cut& cut) const {  // of this lane's
    u64 sum = 0;
    each<1>(b, e, [&](float v, int i) {
      if (cut.takes(v, i)) sum += w(v);
    });
    return sum;
  }
  __device__ __forceinline__ uint32_t place_q(float v) const {
    const float y = weight::product(m - v, w.ch);
    return y >= 0.f ? ~__float2uint_rz(y * 67108864.f) : 0u;  // 2^26; saturates (NaN: 0 times infinity)
  }
  __device__ __forceinline__ void barrier() const {
    if (split > 1)
      cluster_barrier();
    else
      __syncthreads();
  }
  // Lists of all parts into s.key (a barrier after they were filled).
  __device__ void collect(const List& l) {
    // (a warp a part; where its ids go from the parts' counts)
    const int n = lane < split ? (int)min(remote32(&l.n, lane), (uint32_t)kList) : 0;
    int end = n;
#pragma unroll
    for (int o = 1; o < kMaxSplit; o <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, end, o);
      if (lane >= o) end += t;
    }
    static_assert(kWarps >= kMaxSplit, "a warp a part");
    const int mine = __shfl_sync(0xffffffffu, n, warp), at = __shfl_sync(0xffffffffu, end, warp) - mine;
    for (int i = lane; i < mine && at + i < kList; i += 32) s.key[at + i] = remote64(&l.key[i], warp);
    if (warp == 0 && lane == kMaxSplit - 1) s.n_key = min(end, kList);
    __syncthreads();
  }
  __device__ __forceinline__ void push(List& l, u64 k) {
    const uint32_t at = atomicAdd(&l.n, 1u);
    if (at < kList) l.key[at] = k;
  }

  // s.bin: the bin, from the largest down, at which the cluster's running sum over
  // the histograms h reaches the goal from `before` on (bin 0 if none does); what
  // is in front of it, its ids, and this part's.  Of the groups of 32 bins first,
  // then of its group's (all bins of all parts took 6000 clocks: 64 KB a CTA from
  // others').  *own: this part's sum in bin kBins - 1 - tid.  Warp 0 has the
  // results (the others after a barrier).
  template <bool MASS, typename Goal>
  __device__ __forceinline__ void reach_bin(const uint32_t (*h)[kBins], int parity, u64 before, bool first_digit, u64* goal, Goal goal_of,
                                            u64* own) {
    const int mine = kBins - 1 - tid;  // (the largest first)
    *own = MASS ? h[1][mine] + ((u64)h[2][mine] << 16) + ((u64)h[3][mine] << 32) : h[0][mine];
    const u64 own32 = warp_sum64(*own);
    if (lane == 0) s.group[parity][warp] = own32;
    barrier();
    {
      const u64 x = warp_sum64(lane < split ? remote64(&s.group[parity][warp], lane) : 0);
      if (lane == 0) s.red[warp] = x;
    }
    __syncthreads();
    const u64 of_group = lane < kWarps ? s.red[lane] : 0, upto = before + warp_scan64(of_group, lane);
    if (first_digit) *goal = goal_of(__shfl_sync(0xffffffffu, upto, 31));
    const unsigned reach = __ballot_sync(0xffffffffu, upto >= *goal);
    const int g = min(reach ? __ffs(reach) - 1 : 31, kWarps - 1);
    const int bin = kBins - 1 - (g * 32 + lane);
    if (warp < split) {  // (a warp a part)
      s.of_bin[warp][lane] = MASS ? remote32(&h[1][bin], warp) + ((u64)remote32(&h[2][bin], warp) << 16) + ((u64)remote32(&h[3][bin], warp) << 32) : 0;
      s.in_bin[warp][lane] = remote32(&h[0][bin], warp);
    }
    __syncthreads();
    if (warp == 0) {
      const u64 front = __shfl_sync(0xffffffffu, upto - of_group, g);
      u64 sum = 0;
      uint32_t count = 0;
      for (int r = 0; r < split; ++r) {
        sum += s.of_bin[r][lane];
        count += s.in_bin[r][lane];
      }
      if (!MASS) sum = count;
      const u64 inc = front + warp_scan64(sum, lane);
      const unsigned it = __ballot_sync(0xffffffffu, reaches(*goal, inc - sum, sum));
      if (lane == (it ? __ffs(it) - 1 : 31)) {
        s.bin = bin;
        s.before = inc - sum;
        s.count = count;
        s.own = h[0][bin];
      }
    }
  }

  // The largest key at which the running sum (ids that `least` takes, from the
  // largest key down) of counts, or weights (MASS), reaches the goal;
  // goal_of(total) gives it from the sum of all.  With MASS s.mass is then this
  // part's sum of the weights from the cut on.
  template <bool MASS, typename Goal>
  __device__ u64 find_cut(const Cut least, Goal goal_of) {
    Place want{0, 0, 0}, mask{0, 0, 0};
    u64 before = 0, goal = 0;
    List& list = s.list[MASS];
    // the ids that agree in the digits so far have a logit in [lo, hi]
    float lo = least.v, hi = INFINITY;
    auto agrees = [&](float v, int i, int level) {
      if (!(v >= lo && v <= hi) || !least.takes(v, i)) return false;
      // (what fills the vectors is nobody's; weights of 0 would only crowd the others)
      if (MASS ? !(weight::product(m - v, w.ch) < 46.f) : i < id0 || i >= id1) return false;
      return level < 5 || !(((order_bits(v) ^ want.o) & mask.o) | (((0xfffffu - (uint32_t)i) ^ want.i) & mask.i));
    };
    int level = 0;
    for (;; ++level) {
      const int shift = shift_of(level), bits = bits_of(level);
      uint32_t(*h)[kBins] = s.hist[level & 1];
#pragma unroll
      for (int j = 0; j < (MASS ? 4 : 1); ++j) h[j][tid] = 0;
      if (tid == 0) s.n_few = 0;
      __syncthreads();
      auto add = [&](float v, int i) {
        const uint32_t field = level < 4 ? place_q(v) : level < 8 ? order_bits(v) : 0xfffffu - (uint32_t)i;
        const uint32_t bin = (field >> shift) & ((1u << bits) - 1);
        if constexpr (MASS) {
          const u64 k = w(v);
          atomicAdd(&h[0][bin], 1u);
          atomicAdd(&h[1][bin], (uint32_t)k & 0xffffu);
          if (k >> 16) atomicAdd(&h[2][bin], (uint32_t)(k >> 16) & 0xffffu);
          if (k >> 32) atomicAdd(&h[3][bin], (uint32_t)(k >> 32));
        } else {
          atomicAdd(&h[0][bin], 1u);
        }
      };
      if (MASS && level == 0 && least.v == -INFINITY) {  // (every id)
        each<1>(i0, i1, [&](float v, int i) {
          if (weight::product(m - v, w.ch) < 46.f) add(v, i);
        });
      } else if (level == 0 || s.own > kGather) {
        each<1>(i0, i1, [&](float v, int i) {
          if (agrees(v, i, level)) add(v, i);
        });
      } else {
        // few ids, brought together first (a weight takes a warp the same time for one lane's)
        each<2>(i0, i1, [&](float v, int i) {
          if (agrees(v, i, level)) {
            const uint32_t at = atomicAdd(&s.n_few, 1u);
            if (at < kGather) s.few[at] = key_of(v, i);  // (no more than were counted, if logits stay as they are)
          }
        });
        __syncthreads();
        for (int i = tid; i < (int)min(s.n_few, (uint32_t)kGather); i += kThreads) {
          const Cut c = cut_of(s.few[i]);
          add(c.v, (int)c.id);
        }
      }
      __syncthreads();
      u64 own;
      reach_bin<MASS>(h, level & 1, before, level == 0, &goal, goal_of, &own);
      if (warp == 0) {
        __syncwarp();
        if (level < 4) {
          // the logits of that bin, by a search 16 ways at once on each side
          const uint32_t digits = want.q | (uint32_t)s.bin << shift, dm = mask.q | ((1u << bits) - 1) << shift;
          uint32_t at = 0;  // ordered logits: the largest with a place below, or (upper lanes) not above
          for (int step = 28; step >= 0; step -= 4) {
            const uint32_t x = at + ((uint32_t)(lane & 15) << step);
            const uint32_t q = place_q(fminf(value_of(x), m)) & dm;
            const bool less = lane < 16 ? q < digits : q <= digits;
            const bool nan = x < 0x007fffffu, up = x > 0xff800000u;  // (NaN's patterns: below and above all logits)
            const unsigned yes = __ballot_sync(0xffffffffu, (lane & 15) == 0 || nan || (!up && less));
            at += (uint32_t)(31 - __clz((lane < 16 ? yes : yes >> 16) & 0xffffu)) << step;
          }
          if (lane == 0) s.lo = value_of(max(at, 0x007ffffeu) + 1);
          if (lane == 16) s.hi = value_of(min(max(at, 0x007fffffu), 0xff800000u));
        }
      }
      __syncthreads();
      before = s.before;
      if (level < 4) {
        lo = fmaxf(s.lo, least.v);
        hi = s.hi;
      }
      if constexpr (MASS) {  // this part's weights in the bins in front
        const u64 mass = warp_sum64(kBins - 1 - tid > s.bin ? own : 0);
        if (lane == 0 && mass) atomicAdd(&s.mass, mass);
      }
      const uint32_t digit = (uint32_t)s.bin << shift, dm = ((1u << bits) - 1) << shift;
      uint32_t& wf = level < 4 ? want.q : level < 8 ? want.o : want.i;
      uint32_t& mf = level < 4 ? mask.q : level < 8 ? mask.o : mask.i;
      wf |= digit;
      mf |= dm;
      if (s.count <= kList || level == kLevels - 1) break;  // (a bin of the last digit is one id)
    }
    // the ids left, one against another
    each<2>(i0, i1, [&](float v, int i) {
      if (agrees(v, i, kLevels)) push(list, key_of(v, i));
    });
    barrier();
    collect(list);
    const int n = s.n_key;
    u64 k = 0, v = 0;
    if (tid < n) {
      k = s.key[tid];
      v = MASS ? w(value_of((uint32_t)(k >> 32))) : 1;
      s.wt[tid] = v;
    }
    __syncthreads();
    if (tid < n) {
      u64 front = before;
      for (int j = 0; j < n; ++j)
        if (s.key[j] > k) front += s.wt[j];
      if (reaches(goal, front, v)) s.cut = k;
    }
    __syncthreads();
    if (MASS && tid < (int)list.n) {
      const u64 mine = list.key[tid];
      if (mine >= s.cut) atomicAdd(&s.mass, w(value_of((uint32_t)(mine >> 32))));
    }
    return s.cut;
  }
};

// u 2^64 of u in [0, 1), what is below 1 dropped.
__device__ __forceinline__ u64 fixed64(float u) {
  const uint32_t b = __float_as_uint(u);
  const int e = (int)(b >> 23) - 86;
  const u64 f = (b & 0x7fffffu) | 0x800000u;
  return e >= 0 ? f << e : e > -24 ? f >> -e : 0;
}
// floor(u S), and top_p S rounded up (1 at least).
__device__ __forceinline__ u64 share(float u, u64 S) { return __umul64hi(fixed64(u), S); }
__device__ __forceinline__ u64 share_up(float p, u64 S) {
  const u64 f = p > 0.f ? fixed64(p) : 0;
  return max(1ull, __umul64hi(f, S) + (f * S != 0));
}

// Row r's settings.
struct Set {
  float temp, tp, mp;
  int k;
  __device__ __forceinline__ Set(const SampleArgs& a, int r) {
    temp = a.set.d_temperature ? a.set.d_temperature[r] : a.set.temperature;
    k = a.set.d_top_k ? a.set.d_top_k[r] : a.set.top_k;
    tp = a.set.d_top_p ? a.set.d_top_p[r] : a.set.top_p;
    mp = a.set.d_min_p ? a.set.d_min_p[r] : a.set.min_p;
  }
  // 0: one or two readings of the row, 1: its weights too, 2: cuts by digits
  __device__ __forceinline__ int cost(int V) const {
    const bool has_k = k >= 1 && k < V;
    return !(temp > 0.f) || (has_k && k <= kFew) ? 0 : has_k || tp < 1.f ? 2 : 1;
  }
};

// The i-th row when those that cost most come first (of one cost: by threads).
__device__ int costly_first(const SampleArgs& a, Shared& s, int i, int tid) {
  const int lane = tid & 31, warp = tid >> 5;
  u64 mine = 0;  // rows of this thread by cost, 20 bits each, the costliest lowest
  for (int r = tid; r < a.rows; r += kThreads) mine += 1ull << (20 * (2 - Set(a, r).cost(a.V)));
  const u64 upto = warp_scan64(mine, lane);
  if (lane == 31) s.red[warp] = upto;
  __syncthreads();
  u64 all = 0, front = upto - mine;
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) front += s.red[w];
    all += s.red[w];
  }
  auto of = [](u64 x, int c) { return (int)(x >> (20 * c) & 0xfffff); };
  int c = 0;
  while (c < 2 && i >= of(all, c)) i -= of(all, c++);
  i -= of(front, c);
  if (i >= 0 && i < of(mine, c))
    for (int r = tid; r < a.rows; r += kThreads)
      if (2 - Set(a, r).cost(a.V) == c && i-- == 0) s.bin = r;
  __syncthreads();
  return (int)min((unsigned)s.bin, (unsigned)a.rows - 1u);
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 2)
    k_sample(const __grid_constant__ SampleArgs a, const __grid_constant__ Pow2Table pow2, int split, bool order) {
  __shared__ Shared s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, V = a.V;
  const int place = blockIdx.x / split, part = blockIdx.x - place * split;
  const int row = order ? costly_first(a, s, place, tid) : place;
  if (tid == 0) s.row = row;  // (read from here on: a register less)

  // this part's ids, in whole vectors of 16 bytes
  constexpr int VE = Vec<T>::kN;
  const int v0 = (int)((long long)V * part / split), v1 = (int)((long long)V * (part + 1) / split), n = v1 - v0;
  const T* src = static_cast<const T*>(a.x) + (long long)row * a.ld + v0;
  const int off = (int)((reinterpret_cast<uintptr_t>(src) & 15) / sizeof(T));  // (elements)
  const int nvec = (off + n + VE - 1) / VE;
  if (tid < 64) s.table[tid] = pow2.t[tid];
  if (tid < 2) s.list[tid].n = 0;
  if (tid == 0) s.mass = 0;
  const Set set(a, row);
  const float temp = set.temp, tp = set.tp, mp = set.mp;
  const int k = set.k;
  const float u = fminf(fmaxf(a.u[row], 0.f), 1.f - 5.9604644775390625e-8f);
  // (one thread, in 64 bits, which all threads at once would wait for)
  if (tid == kThreads - 1) {
    const weight::Rate c = weight::rate_of(temp);
    s.ch = c.h;
    s.cl = c.l;
    s.span = mp > 0.f ? fmin((double)temp, 3.4028234663852886e38) * log((double)mp) : 0.0;
  }
  __syncthreads();

  const int seg = (nvec + kWarps - 1) / kWarps;
  Row<T> r{s, src - off, off, off + n, v0 - off, v0, v1, min(nvec, warp * seg), min(nvec, (warp + 1) * seg), split, tid, lane, warp,
           0.f, Weight{}};
  // the largest logit (the lowest id of equal ones)
  uint32_t top = 0;
  int top_i = 0;
  r.template each<4>(r.i0, r.i1, [&](float v, int i) {
    const uint32_t o = order_bits(v);
    if (o > top) {
      top = o;
      top_i = i;
    }
  });
  u64 best = top ? ((u64)top << 32) | (0xffffffffu - (uint32_t)top_i) : 0;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) best = max(best, __shfl_xor_sync(0xffffffffu, best, o));
  if (lane == 0) s.red[warp] = best;
  __syncthreads();
  for (int j = 0; j < kWarps; ++j) best = max(best, s.red[j]);
  if (split > 1) {
    if (tid == 0) s.best = best;
    cluster_barrier();
    u64 x = lane < split ? remote64(&s.best, lane) : 0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x = max(x, __shfl_xor_sync(0xffffffffu, x, o));
    best = x;
  }
  const float m = value_of((uint32_t)(best >> 32));
  if (!(fabsf(m) < INFINITY) || !(temp > 0.f)) {
    if (part == 0 && tid == 0) {
      a.token[s.row] = m == -INFINITY ? 0 : (int)(0xffffffffu - (uint32_t)best);
      if (a.logprob) a.logprob[s.row] = fabsf(m) < INFINITY ? 0.f : NAN;
    }
    if (split > 1) cluster_barrier();
    return;
  }
  r.m = m;
  r.w = Weight{m, s.ch, s.cl, smem_u32(s.table)};
  if (mp > 0.f) {
    if (tid == 0) {
      const double b = (double)m + s.span;
      const float f = (float)b;
      s.least = (double)f < b ? nextafterf(f, INFINITY) : f;
    }
    __syncthreads();
  }
  const float least = mp > 0.f ? s.least : -INFINITY;
  const bool has_k = k >= 1 && k < V;

  if (has_k && k <= kFew) {
    // Few ids: a bin of -log2 of the weight such that k threads' largest logits
    // reach it; the ids that do are no fewer.
    uint32_t* h = s.hist[0][0];
    h[tid] = 0;
    __syncthreads();
    const uint32_t mine = r.place_q(value_of(top)) >> 23;
    if (top) atomicAdd(&h[mine], 1u);
    u64 goal = k, own;
    r.template reach_bin<false>(s.hist[0], 0, 0, false, &goal, [](u64 x) { return x; }, &own);
    __syncthreads();
    const uint32_t from = (uint32_t)s.bin;
    if (top && mine >= from)
      r.template each<2>(r.i0, r.i1, [&](float v, int i) {
        if (r.place_q(v) >> 23 >= from) r.push(s.list[0], key_of(v, i));
      });
    r.barrier();
    const uint32_t all = __reduce_add_sync(0xffffffffu, lane < split ? remote32(&s.list[0].n, lane) : 0u);
    if (all <= kList) {
      if (part == 0) {
        r.collect(s.list[0]);
        const int cnt = s.n_key;
        u64 key = 0, v = 0;
        float x = 0.f;
        int rank = 0;
        if (tid < cnt) {
          key = s.key[tid];
          x = value_of((uint32_t)(key >> 32));
          for (int j = 0; j < cnt; ++j) rank += s.key[j] > key;
          v = rank < k ? r.w(x) : 0;
          s.wt[tid] = v;
        }
        __syncthreads();
        bool keep = tid < cnt && rank < k && (rank == 0 || x >= least);
        u64 sum = 0, front_w = 0;
        if (tid < cnt) {
          for (int j = 0; j < cnt; ++j) {
            sum += s.wt[j];
            if (s.key[j] > key) front_w += s.wt[j];
          }
          if (tp < 1.f && rank > 0) keep = keep && front_w < share_up(tp, sum);
        }
        __syncthreads();
        if (tid < cnt) s.wt[tid] = keep ? v : 0;
        __syncthreads();
        if (tid < cnt) {
          const uint32_t id = (uint32_t)key;  // (~id)
          u64 total = 0, upto = 0;
          for (int j = 0; j < cnt; ++j) {
            total += s.wt[j];
            if ((uint32_t)s.key[j] > id) upto += s.wt[j];
          }
          const u64 goal = share(u, total);
          if (keep && upto <= goal && goal < upto + v) {
            a.token[s.row] = (int)(0xffffffffu - id);
            if (a.logprob) a.logprob[s.row] = logf((float)v / (float)total);
          }
        }
      }
      if (split > 1) cluster_barrier();
      return;
    }
    r.barrier();
    if (tid == 0) s.list[0].n = 0;
    __syncthreads();
  }

  u64 cut = 0;
  if (has_k) cut = r.template find_cut<false>(cut_of(0), [&](u64) { return (u64)k; });
  bool known = false;  // s.mass holds the weights kept
  if (tp < 1.f) {
    cut = r.template find_cut<true>(cut_of(cut), [&](u64 S) { return share_up(tp, S); });
    known = true;
  }
  if (mp > 0.f && ((u64)order_bits(least) << 32) > cut) {
    cut = (u64)order_bits(least) << 32;
    known = false;
  }
  cut = min(cut, best);
  const Cut keep = cut_of(cut);
  // the weights of each warp's segment
  auto segments = [&] {
    const u64 sum = warp_sum64(r.mass(r.i0, r.i1, keep));
    if (lane == 0) s.sums[warp] = sum;
    __syncthreads();
  };
  if (!known) {
    segments();
    if (tid == 0) {
      u64 sum = 0;
      for (int j = 0; j < kWarps; ++j) sum += s.sums[j];
      s.mass = sum;
    }
  }
  // and of each part: in front of this one's, this one's, all
  r.barrier();
  const u64 of_part = lane < split ? remote64(&s.mass, lane) : 0;
  const u64 all = warp_sum64(of_part);
  const u64 goal = share(u, all);
  // The part it is in; with its segments' sums at hand that part's CTA finds the
  // id, else all take a share of it first (one alone took 35,000 clocks).
  u64 upto = of_part;
#pragma unroll
  for (int o = 1; o < kMaxSplit; o <<= 1) {
    const u64 t = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += t;
  }
  const int owner = max(__ffs(__ballot_sync(0xffffffffu, lane < split && upto > goal)), 1) - 1;
  u64 front = __shfl_sync(0xffffffffu, upto - of_part, owner);
  const int o0 = (int)((long long)V * owner / split), o1 = (int)((long long)V * (owner + 1) / split);
  const T* osrc = static_cast<const T*>(a.x) + (long long)s.row * a.ld + o0;
  const int ooff = (int)((reinterpret_cast<uintptr_t>(osrc) & 15) / sizeof(T)), ovec = (ooff + o1 - o0 + VE - 1) / VE;
  r.x = osrc - ooff;
  r.off = ooff;
  r.end = ooff + o1 - o0;
  r.first = o0 - ooff;
  int base = 0, width = kWarps * ((ovec + kWarps - 1) / kWarps);  // this CTA's vectors of it
  bool mine = part == owner;
  if (known) {
    const int each = (ovec + split * kWarps - 1) / (split * kWarps);  // a warp's
    base = part * kWarps * each;
    width = kWarps * each;
    const u64 sum = warp_sum64(r.mass(min(ovec, base + warp * each), min(ovec, base + (warp + 1) * each), keep));
    if (lane == 0) s.sums[warp] = sum;
    __syncthreads();
    const u64 total = warp_sum64(lane < kWarps ? s.sums[lane] : 0);
    if (tid == 0) s.best = total;  // (its last use is long past)
    r.barrier();
    const u64 x = lane < split ? remote64(&s.best, lane) : 0;
    front += warp_sum64(lane < part ? x : 0);
    mine = front <= goal && goal < front + total;
  }
  if (mine) {
    // the segment it is in, then the sixteenth of that, then the id
    const int step = width / kWarps;
    int ow = 0;
    while (ow < kWarps - 1 && front + s.sums[ow] <= goal) front += s.sums[ow++];
    const int s0 = min(ovec, base + ow * step), s1 = min(ovec, s0 + step), sub = (s1 - s0 + kWarps - 1) / kWarps;
    auto range = [&](int j, int* b, int* e) {
      *b = min(s1, s0 + j * sub);
      *e = min(s1, *b + sub);
    };
    int b, e;
    range(warp, &b, &e);
    const u64 sum = warp_sum64(r.mass(b, e, keep));
    if (lane == 0) s.red[warp] = sum;
    __syncthreads();
    int os = 0;
    while (os < kWarps - 1 && front + s.red[os] <= goal) front += s.red[os++];
    if (warp == 0) {
      range(os, &b, &e);
      for (int i = b; i < e; i += 32) {
        u64 w[VE] = {}, x = 0;
        if (i + lane < e) {
          const Vec<T> v(r.load(i + lane));
#pragma unroll
          for (int j = 0; j < VE; ++j) x += w[j] = keep.takes(v.v[j], r.id(i + lane, j)) ? r.w(v.v[j]) : 0;
        }
        const u64 inc = warp_scan64(x, lane);
        const unsigned hit = __ballot_sync(0xffffffffu, front + inc > goal);
        if (hit) {
          if (lane == __ffs(hit) - 1) {
            u64 at = front + inc - x;
            int pick = 0;  // elements whose sums do not exceed the goal
#pragma unroll
            for (int j = 0; j < VE; ++j) {
              at += w[j];
              pick += at <= goal;
            }
            u64 weight = w[0];
#pragma unroll
            for (int j = 1; j < VE; ++j) weight = j == pick ? w[j] : weight;
            a.token[s.row] = r.id(i + lane, pick);
            if (a.logprob) a.logprob[s.row] = logf((float)weight / (float)all);
          }
          break;
        }
        front += __shfl_sync(0xffffffffu, inc, 31);
      }
    }
  }
  if (split > 1) cluster_barrier();  // nobody leaves while its shared memory may still be read
}

// Settings that differ from row to row.
bool of_each(const rl_sampling& s) { return s.d_temperature || s.d_top_k || s.d_top_p || s.d_min_p; }

// CTAs a row is split over: as many as its parts' sums need, and twice as many
// while, before that, they are no more than the SMs and a part keeps 4096 ids (so up
// to two CTAs an SM, which all are at work at once: 64 rows of
// 128,256 cut by mass: 72 us in 4 parts, 88 in 2, 91 in 8; 500 of 50,257: 211 whole,
// 207 in halves; one row: 14.4 us in 16); while they are no more than twice the
// SMs where rows' settings differ and the costliest take the time (48 rows of
// 50,257: 39 us in 8, 44 in 4; 200: 58 in halves, 112 whole; 64 of 128,256: 48 in
// 8, 55 in 4); and halves of long rows while there are no more than four rows an
// SM, which start in turn (320 of 50,257: 72 us, 98 whole; 500: 104 and 110; even
// at the end, 608: 124 and 121; of 20,011 ids 400 are slower so, 63 and 55).
int pick_split(int rows, int V, bool each, int sms) {
  int s = 1;
  auto more = [&] {
    const long long ctas = (long long)rows * s;
    return V > 4096 * s && ctas <= (each ? s == 1 && V > 32768 ? 4ll : 2ll : 1ll) * sms;
  };
  while (s < kMaxSplit && (V > kMostIds * s || more())) s *= 2;
  return s;
}

template <typename T>
cudaError_t launch(const SampleArgs& a, const Pow2Table& table, cudaStream_t st) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = device_sm_count(dev, &sms);
  if (e != cudaSuccess) return e;
  auto kern = k_sample<T>;
  {
    static std::mutex mu;
    static bool done[kOpDevices] = {};
    std::lock_guard<std::mutex> lock(mu);
    if (!done[dev]) {
      e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
      if (e != cudaSuccess) return e;
      done[dev] = true;
    }
  }
  const int split = pick_split(a.rows, a.V, of_each(a.set), sms);
  if ((long long)a.rows * split >= 1ll << 31) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.rows * split);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = split;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // Rows of different cost that do not all fit at once: the last to start should
  // be the shortest (500 of 50,257 in halves: 104 us, 116 as they come; 500 of
  // 128,256: 168 and 221; 600 of 9,001: 59 and 52, so rows of some length only).
  const bool order = of_each(a.set) && a.V > 16384 && a.rows <= kOrder && (long long)a.rows * split > 2ll * sms;
  return cudaLaunchKernelEx(&cfg, kern, a, table, split, order);
}

}  // namespace

cudaError_t launch_sample(const SampleArgs& a, cudaStream_t s) {
  static const Pow2Table table = [] {
    Pow2Table t;
    for (int j = 0; j < 64; ++j) t.t[j] = weight::entry(j);
    return t;
  }();
  if (a.dtype == RL_DT_F32) return launch<float>(a, table, s);
  if (a.dtype == RL_DT_BF16) return launch<bf16>(a, table, s);
  return launch<__half>(a, table, s);
}

}  // namespace river

using namespace river;

// Whether n bytes from p on meet one of `rows` rows of `len` bytes, `step` apart, from x on.
static bool meets(const void* p, uint64_t n, const void* x, int rows, uint64_t len, uint64_t step) {
  const uint64_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(x);
  if (a < b) return n > b - a;
  const uint64_t row = (a - b) / step, in = (a - b) % step;
  return row < (uint64_t)rows && (in < len || (row + 1 < (uint64_t)rows && n > step - in));
}

extern "C" rl_status rl_sample(const void* d_logits, int32_t dtype, int32_t rows, int32_t vocab, int64_t row_stride,
                               const float* d_u, const rl_sampling* settings, int32_t* d_token, float* d_logprob,
                               rl_stream_t stream) {
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
  const uint64_t n = 4ull * rows, width = dtype == RL_DT_F32 ? 4 : 2, apart = (uint64_t)row_stride < 1ull << 60 ? row_stride : 1ull << 60;
  for (const void* out : {(const void*)d_token, (const void*)d_logprob}) {
    bool hit = out && meets(out, n, d_logits, rows, width * vocab, width * apart);
    for (const void* x : {(const void*)d_u, (const void*)s.d_temperature, (const void*)s.d_top_k, (const void*)s.d_top_p, (const void*)s.d_min_p})
      hit = hit || (out && x && meets(out, n, x, 1, n, n));
    if (hit) return bad(RL_ERR_INVALID_ARG, "an output overlaps an input");
  }
  if (d_logprob && meets(d_token, n, d_logprob, 1, n, n)) return bad(RL_ERR_INVALID_ARG, "the outputs overlap");
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
  const cudaError_t e = launch_sample(a, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return set_error(RL_ERR_CUDA, cudaGetErrorString(e));
  return RL_OK;
}
