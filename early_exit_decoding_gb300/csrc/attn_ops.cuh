// What the stand-alone attention operators' kernels share: lengths, 16-bit
// element pairs, the row-by-row form, tensor maps of caller-owned caches.
#pragma once

#include <float.h>
#include <math.h>

#include "dev_common.cuh"
#include "internal.h"

namespace river {
namespace attn {

template <bool F16>
__device__ __forceinline__ float2 unpack2(uint32_t v) {
  if constexpr (F16)
    return __half22float2(*reinterpret_cast<const __half2*>(&v));
  else
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&v));
}
template <bool F16>
__device__ __forceinline__ uint32_t pack2(float x, float y) {
  if constexpr (F16) {
    const __half2 h = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Length of sequence b, clamped to the rows laid out for it.
struct Lens {
  int n, ql;  // token rows of a sequence, query rows among them
};
__device__ __forceinline__ Lens seq_lens(const AttnOpArgs& a, int b, bool report) {
  // (both loads before either check, which may write the error word)
  const int kv = a.kv_len ? __ldg(a.kv_len + (long long)b * a.kv_len_step) : 0, q = a.q_len ? __ldg(a.q_len + b) : a.Tq;
  const long long n = (long long)kv + a.kv_len_add;
  if (report && a.err && (n < 0 || n > a.cap || q < 0 || q > a.Tq)) atomicOr(a.err, RL_DEVERR_CAPACITY);
  return Lens{(int)max(0ll, min(n, (long long)a.cap)), max(0, min(q, a.Tq))};
}

// One row in the plain form, held by a warp: lane has dims 2 * lane + 64 * i,
// i < HD / 64; one key at a time with a running maximum and sum.  Keys the
// row does not see are skipped, never multiplied by a zero weight.
template <int HD, bool F16>
struct RowAcc {
  float2 q[HD / 64], o[HD / 64];
  float m = -INFINITY, l = 0.f;
  __device__ __forceinline__ void load_q(const AttnOpArgs& a, int b, int t, int h, int lane) {
    const long long at = b * a.qs[0] + t * a.qs[1] + h * a.qs[2] + 2 * lane;
#pragma unroll
    for (int i = 0; i < HD / 64; ++i) {
      if (a.q_f32) {
        const float2 f = *reinterpret_cast<const float2*>(static_cast<const float*>(a.q) + at + 64 * i);
        q[i] = unpack2<F16>(pack2<F16>(f.x, f.y));
      } else {
        q[i] = unpack2<F16>(*reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(a.q) + at + 64 * i));
      }
      o[i] = make_float2(0.f, 0.f);
    }
  }
  __device__ __forceinline__ void keys(const KeySrc& s, int b, int hk, int j0, int j1, float scale, int lane) {
    const long long kb = b * s.ks[0] + hk * s.ks[1] + 2 * lane, vb = b * s.vs[0] + hk * s.vs[1] + 2 * lane;
    for (int j = j0; j < j1; ++j) {
      float d = 0.f;
      uint32_t vv[HD / 64];
#pragma unroll
      for (int i = 0; i < HD / 64; ++i) {
        const float2 k = unpack2<F16>(
            *reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(s.k) + kb + j * s.ks[2] + 64 * i));
        vv[i] = *reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(s.v) + vb + j * s.vs[2] + 64 * i);
        d += q[i].x * k.x + q[i].y * k.y;
      }
      d = dev::warp_sum(d) * scale;
      const float mn = fmaxf(m, d), mu = mn == -INFINITY ? 0.f : mn;
      const float c = __expf(m - mu), e = __expf(d - mu);
      l = l * c + e;
#pragma unroll
      for (int i = 0; i < HD / 64; ++i) {
        const float2 v = unpack2<F16>(vv[i]);
        o[i].x = o[i].x * c + e * v.x;
        o[i].y = o[i].y * c + e * v.y;
      }
      m = mn;
    }
  }
  // Every key that query row t of sequence b, of n rows and ql queries, sees (its first key at `base`).
  __device__ __forceinline__ void window(const AttnOpArgs& a, int b, int t, int hk, int n, int ql, int lane, int base) {
    const int p = n - ql + t, lo = max(0, p - a.window + 1);
    keys(a.kv, b, hk, base, base + min(min(a.sinks, lo), p + 1), a.scale, lane);
    keys(a.kv, b, hk, base + lo, base + p + 1, a.scale, lane);
  }
  __device__ __forceinline__ void store(const AttnOpArgs& a, int b, int t, int h, int lane) {
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const long long at = b * a.os[0] + t * a.os[1] + h * a.os[2] + 2 * lane;
#pragma unroll
    for (int i = 0; i < HD / 64; ++i)
      *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + at + 64 * i) =
          pack2<F16>(o[i].x * inv, o[i].y * inv);
    if (lane == 0 && a.lse)
      a.lse[((long long)b * a.Tq + t) * a.Hq + h] = l == 0.f ? -INFINITY : m + logf(l);
  }
};

template <int HD, bool F16>
__device__ __noinline__ void exact_row(const AttnOpArgs& a, int b, int t, int h, int n, int ql, int lane, int base = 0) {
  RowAcc<HD, F16> r;
  r.load_q(a, b, base + t, h, lane);
  r.window(a, b, t, h / (a.Hq / a.Hkv), n, ql, lane, base);
  r.store(a, b, base + t, h, lane);
}

// Division of n < 2^31 by a fixed d >= 1 as a multiplication and a shift (a
// division takes some 130 clocks, and a CTA's first copy waits for several in
// a row): with l = ceil(log2 d) and m = floor(2^32 (2^l - d) / d) + 1,
// n / d = (mulhi(m, n) + n) >> l (Granlund and Montgomery 1994).
struct FastDiv {
  uint32_t m, l;
  int d;
  FastDiv() = default;
  explicit FastDiv(int div) : m(0), l(0), d(div) {
    while ((1ll << l) < div) ++l;
    m = (uint32_t)(((1ull << 32) * ((1ull << l) - (unsigned long long)div)) / (unsigned long long)div + 1);
  }
  __device__ __forceinline__ int quot(int n) const { return (int)((__umulhi(m, (uint32_t)n) + (uint32_t)n) >> l); }
};

// The tile of `rows` rows that comes `rank`-th when packed sequences' tiles (of
// their rows x rep; at most `most` rows of a sequence count, of the N laid out)
// are taken from the last of the longest on, since a later tile of a prompt sees
// more keys; false: there are no more.  The tiles numbered L or more are
// f(L) = sum_b max(0, n_b - L), so the number is the L with
// f(L + 1) <= rank < f(L).  The same for every lane.
struct RowTile {
  int seq, first, n, number;  // the sequence, its first row and rows; which of its tiles
};
__device__ __forceinline__ bool row_tile(const int* start, int B, int N, int most, int rep, int rows, int rank, int lane, RowTile* t) {
  auto span = [&](int b, int* first) {
    if (b >= B) return 0;
    const int s0 = __ldg(start + b), s1 = __ldg(start + b + 1);
    *first = max(0, min(s0, N));
    return min(max(0, min(s1, N) - *first), most);
  };
  auto tiles_of = [&](int b) {
    int first;
    return (int)(((long long)span(b, &first) * rep + rows - 1) / rows);
  };
  const int own = tiles_of(lane);
  auto above = [&](int L) {  // f(L); at most 2^30, which only starts that overlap pass
    int n = min(max(0, own - L), 1 << 25);
    for (int b = 32 + lane; b < B; b += 32) n = min(n + max(0, tiles_of(b) - L), 1 << 25);
    return (int)__reduce_add_sync(0xffffffffu, n);
  };
  int top = own;
  for (int b = 32 + lane; b < B; b += 32) top = max(top, tiles_of(b));
  int lo = 0, hi = __reduce_max_sync(0xffffffffu, top);
  if (rank >= above(0)) return false;
  while (hi - lo > 1) {  // f(lo) > rank >= f(hi)
    const int mid = (lo + hi) >> 1;
    if (above(mid) > rank)
      lo = mid;
    else
      hi = mid;
  }
  rank -= above(hi);
  t->number = lo;
  for (int b0 = 0; b0 < B; b0 += 32) {
    const unsigned has = __ballot_sync(0xffffffffu, (b0 ? tiles_of(b0 + lane) : own) > lo);
    const int n = __popc(has);
    if (rank < n) {
      const unsigned it = __ballot_sync(0xffffffffu, (has >> lane & 1) && __popc(has & ((1u << lane) - 1)) == rank);
      t->seq = b0 + __ffs(it) - 1;
      t->n = span(t->seq, &t->first);
      return true;
    }
    rank -= n;
  }
  return false;  // (not reached)
}

// Tensor maps of one K and one V source: five axes (64 dims, token rows,
// 64-dim blocks, KV heads, sequences), so one copy brings `rows` token rows of
// all dims as HD / 64 blocks of rows x 128 bytes, 128-byte swizzle; rows past
// the last one read as zero.  An axis of stride 0 has extent 1 and its
// coordinate is multiplied by 0.
struct KvMaps {
  CUtensorMap k, v;
  int kb, kh, vb, vh;
};
bool make_kv_maps(KvMaps* m, const KeySrc& s, bool f16, int B, int Hkv, int hd, int tokens, int rows);

__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}
__device__ __forceinline__ void tma_load_5d(void* dst, const CUtensorMap* map, int tok, int head, int seq,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %3, %5, %6}], [%2];" ::"r"(dev::smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(dev::smem_u32(bar)), "r"(0), "r"(tok), "r"(head), "r"(seq)
      : "memory");
}

__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Address of this CTA's shared-memory object in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t cluster_map(uint32_t own, int rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(own), "r"(rank));
  return r;
}
__device__ __forceinline__ uint32_t cluster_addr(const void* p, int rank) { return cluster_map(dev::smem_u32(p), rank); }
__device__ __forceinline__ float cluster_ld(uint32_t at) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ float2 cluster_ld2(uint32_t at) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(at) : "memory");
  return v;
}

__device__ __forceinline__ float4 cluster_ld4(uint32_t at) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(at)
               : "memory");
  return v;
}

// Shared memory to global, a multiple of 16 bytes, in the issuing thread's bulk group.
__device__ __forceinline__ void bulk_s2g(void* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(dev::smem_u32(src)), "r"(bytes)
               : "memory");
}

// The shared-prefix workspace: for every (tile of 256 rows, KV head, split of
// the prefix) the rows' sums of weighted values (16-byte chunk c of row q at
// c ^ (q mod chunks)), then for all of them the rows' largest scores (log2
// units; -infinity: no keys) and sums of weights.
__host__ __device__ inline int prefix_rows(int tiles, long long rows) { return tiles > 1 ? 256 : (int)((rows + 31) / 32 * 32); }
struct PrefixWs {
  float *o, *m, *l;
};
__device__ __forceinline__ PrefixWs prefix_ws(void* ws, int tile, int tiles, int rows, int hk, int Hkv, int part, int split,
                                              int hd) {  // split: parts of a tile and KV head, the own keys' too
  const long long R = prefix_rows(tiles, rows), e = ((long long)tile * Hkv + hk) * split + part;
  float* base = static_cast<float*>(ws);
  float* ml = base + (long long)tiles * Hkv * split * R * hd;
  return PrefixWs{base + e * R * hd, ml + e * 2 * R, ml + (e * 2 + 1) * R};
}

}  // namespace attn

// Few query rows against long key ranges (attn_decode.cu).
cudaError_t launch_attn_decode(const AttnOpArgs& a, bool pdl, cudaStream_t s);
// Many query rows on the tensor cores (attn_rows_tc.cu): a prompt's window,
// packed prompts (a.start), or (prefix) every sequence's rows against a.pre into a.ws.
cudaError_t launch_attn_rows_tc(const AttnOpArgs& a, bool prefix, cudaStream_t s);
// Joins the prefix's parts and the own keys' part of every row (attn_decode.cu).
cudaError_t launch_prefix_join(const AttnOpArgs& a, cudaStream_t s);
constexpr int kMaxPrefixSplit = 31;  // and the own keys' part: one a lane
// Whether the own keys' states go to the workspace too and a third launch joins
// all: with more CTAs than the GPU holds at once, those that wait for the
// prefix's products at their end would keep the others from starting.
bool prefix_apart(int B, int rep, int Hkv);
int prefix_split(int B, int rep, int Hkv, int P);
size_t prefix_ws_bytes(int B, int rep, int Hkv, int hd, int P);

}  // namespace river
