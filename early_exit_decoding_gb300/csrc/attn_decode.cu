// Few query rows against long key ranges: single tokens, drafts, and the
// sequences' own keys of a shared-prefix step.
//
// 16 query rows (query position x the heads that share a KV head) form the M
// side of m16n8k16 MMAs; a warp takes units of 16 keys.  Each warp runs its
// own pipeline: lane 0 copies the K and V rows of a unit by TMA into the
// warp's ring (NST stages ahead), the warp waits for them, and keeps a running
// maximum, sum and output of its own units only, so the main loop has no
// barrier between warps.  The keys of a row tile are dealt out unit by unit
// to the warps of a cluster of S CTAs; at the end the warps' states are joined
// through shared memory, the CTAs' through distributed shared memory, in a
// fixed order: no workspace, no atomics, one launch.  Behind a prefix its parts
// are joined at the end too; with many sequences k_prefix_join does that.
//
//   S = q K^T (fp32), w = exp2(S - m) with the running maximum m of the unit's
//   and all earlier keys, l += w in fp32 before w is rounded to the cache's
//   type for O += w V: half a step of the type per weight, the same size as
//   the rounding of the result.
//
// HBM bounds it: 16 keys bring 64 HD bytes and cost HD / 4 MMAs.  64 sequences,
// window 4096, head_dim 128, 8 KV heads: 127 us, 6.4 TB/s, 0.94 of a measured
// copy.  A few sequences are bound by a launch's and a cluster's latency (one
// of 1,024 keys: 6.7 us for 2 MB).
#include <mutex>

#include "attn_ops.cuh"

namespace river {

namespace {

using namespace dev;
using namespace attn;

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kUnit = 16;        // keys a warp takes at a time
constexpr int kRows = 16;        // query rows of a tile
constexpr int kMaxSplit = 12;    // CTAs of a cluster
constexpr unsigned long long kWaitNs = 2000000000ull;  // a wait gives up after two seconds
constexpr float kLog2e = 1.4426950408889634f;

template <int HD>
constexpr int kStageBytes = 2 * kUnit * HD * 2;  // K and V rows of a unit
template <int HD>
constexpr int kStages = HD == 128 ? 2 : 4;  // (with 3 and 6 two CTAs share an SM instead of three:
                                             // 64 ragged 4k windows 143 us, not 128)
template <int HD>
constexpr int kSmem = kWarps * kStages<HD> * kStageBytes<HD> + 1024;

template <bool F16>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    mma_f16(d, a[0], a[1], a[2], a[3], b0, b1);
  else
    mma_bf16(d, a[0], a[1], a[2], a[3], b0, b1);
}

// Query row r of a tile: position row0 + r counts (query, head in group).
struct Tile {
  int b, hk, row0, rep, n, ql;
};
// Divisors of a launch.
struct DecodeShape {
  int split, tiles, presplit, apart;
  FastDiv by_split, by_tiles, by_heads, by_rep;  // CTAs of a cluster, row tiles, KV heads, heads a KV head
};

template <int HD, bool F16>
__device__ __forceinline__ uint32_t load_q2(const AttnOpArgs& a, const Tile& t, const FastDiv& by_rep, int r, int dim) {
  const int i = t.row0 + r, tq = by_rep.quot(i);
  if (tq >= a.Tq) return 0u;
  const long long at = t.b * a.qs[0] + tq * a.qs[1] + (long long)(t.hk * t.rep + i - tq * t.rep) * a.qs[2] + dim;
  if (a.q_f32) {
    const float2 f = *reinterpret_cast<const float2*>(static_cast<const float*>(a.q) + at);
    return pack2<F16>(f.x, f.y);
  }
  return *reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(a.q) + at);
}

template <int HD, bool F16>
__global__ void __launch_bounds__(kThreads, 3)
    k_attn_decode(const __grid_constant__ KvMaps maps, const __grid_constant__ AttnOpArgs a,
                  const __grid_constant__ DecodeShape sh) {
  constexpr int NST = kStages<HD>, SB = kStageBytes<HD>;
  extern __shared__ unsigned char smem_dyn[];
  unsigned char* smem =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~(uintptr_t)1023);
  __shared__ __align__(8) uint64_t full[kWarps][NST];
  __shared__ float s_m[kWarps][kRows], s_l[kWarps][kRows];
  __shared__ float c_m[kRows], c_l[kRows];

  if (threadIdx.x == kThreads - 1) {
    prefetch_map(&maps.k);
    prefetch_map(&maps.v);
  }
  const int split = sh.split, presplit = sh.presplit;
  const int id = sh.by_split.quot(blockIdx.x), head = sh.by_tiles.quot(id);
  const int part = blockIdx.x - id * split;
  Tile t;
  t.rep = sh.by_rep.d;
  t.row0 = (id - head * sh.tiles) * kRows;
  t.b = sh.by_heads.quot(head);
  t.hk = head - t.b * a.Hkv;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const bool report = part == 0 && tid == 0 && t.hk == 0 && t.row0 == 0;
  const Lens len = seq_lens(a, t.b, report);
  t.n = len.n;
  t.ql = len.ql;
  unsigned char* ring = smem + warp * NST * SB;
  if (lane == 0) {
    for (int i = 0; i < NST; ++i) mbar_init(&full[warp][i], 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncwarp();

  // Keys any row of the tile sees: [0, sink_end) and [lo, hi).
  const int t0 = sh.by_rep.quot(t.row0), t1 = min(sh.by_rep.quot(t.row0 + kRows - 1), t.ql - 1);
  const int p0 = max(t.n - t.ql + t0, 0), p1 = t.n - t.ql + t1;
  const bool live = t0 <= t1 && p1 >= 0;
  int lo = live ? max(0, p0 - a.window + 1) : 0;
  const int hi = live ? p1 + 1 : 0;
  int sink_end = min(a.sinks, lo);
  if (sink_end == lo) lo = sink_end = 0;
  const int su = (sink_end + kUnit - 1) / kUnit;
  const int units = su + (hi - lo + kUnit - 1) / kUnit;
  const int W = split * kWarps, first = part * kWarps + warp;
  auto key0 = [&](int u) { return u < su ? u * kUnit : lo + (u - su) * kUnit; };
  auto issue = [&](int u, int st) {
    unsigned char* dst = ring + st * SB;
    mbar_expect_tx(&full[warp][st], SB);
    const int j = key0(u);
    tma_load_5d(dst, &maps.k, j, t.hk * maps.kh, t.b * maps.kb, &full[warp][st]);
    tma_load_5d(dst + SB / 2, &maps.v, j, t.hk * maps.vh, t.b * maps.vb, &full[warp][st]);
  };
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < NST; ++i)
      if (first + i * W < units) issue(first + i * W, i);
  }

  const int g = lane >> 2, c2 = (lane & 3) * 2;
  uint32_t qf[HD / 16][4];
#pragma unroll
  for (int ks = 0; ks < HD / 16; ++ks) {
    qf[ks][0] = load_q2<HD, F16>(a, t, sh.by_rep, g, ks * 16 + c2);
    qf[ks][1] = load_q2<HD, F16>(a, t, sh.by_rep, g + 8, ks * 16 + c2);
    qf[ks][2] = load_q2<HD, F16>(a, t, sh.by_rep, g, ks * 16 + 8 + c2);
    qf[ks][3] = load_q2<HD, F16>(a, t, sh.by_rep, g + 8, ks * 16 + 8 + c2);
  }
  // positions of this thread's two rows
  const int pr0 = t.n - t.ql + sh.by_rep.quot(t.row0 + g), pr1 = t.n - t.ql + sh.by_rep.quot(t.row0 + g + 8);
  const bool one_mask = a.Tq == 1;  // every row sees the same keys
  const float sc = a.scale * kLog2e;

  float o[HD / 8][4];
#pragma unroll
  for (int i = 0; i < HD / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
  float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
  bool ok = true;
  const int mi = lane >> 3, mr = lane & 7;

  // After a wait that gave up nothing is copied or computed any more; the
  // copies already in flight are still waited for (`stop`).
  int st = 0, ph = 0, stop = units;
  for (int u = first; u < stop; u += W) {
    const bool got = mbar_wait_lazy(&full[warp][st], ph, kWaitNs);
    if (!__all_sync(0xffffffffu, got) && ok) {
      ok = false;
      stop = min(units, u + NST * W);
      if (lane == 0 && a.err) atomicOr(a.err, RL_DEVERR_TIMEOUT);
    }
    if (ok) {
      unsigned char* sk = ring + st * SB;
      unsigned char* sv = sk + SB / 2;
      const int j0 = key0(u), cnt = min(kUnit, (u < su ? sink_end : hi) - j0);
      if (cnt < kUnit) {
        // rows behind the range may hold anything: 0 * NaN must not happen
        for (int i = lane; i < (kUnit - cnt) * (HD / 8); i += 32) {
          const int r = cnt + i / (HD / 8), ch = i % (HD / 8);
          *reinterpret_cast<uint4*>(sv + (ch >> 3) * 2048 + r * 128 + (ch & 7) * 16) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        __syncwarp();
      }
      float s[2][4] = {};
      {
        const uint32_t base = smem_u32(sk) + ((mi >> 1) * 8 + mr) * 128;
#pragma unroll
        for (int ks = 0; ks < HD / 16; ++ks) {
          uint32_t kf[4];
          ldsm_x4(kf, base + (ks >> 2) * 2048 + ((((ks & 3) * 2 + (mi & 1)) ^ mr) << 4));
          mma<F16>(s[0], qf[ks], kf[0], kf[1]);
          mma<F16>(s[1], qf[ks], kf[2], kf[3]);
        }
      }
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[nt][e] *= sc;
      if (!one_mask || cnt < kUnit) {
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int jj = nt * 8 + c2 + (e & 1), j = j0 + jj, p = e < 2 ? pr0 : pr1;
            const bool see = jj < cnt && (one_mask || (j <= p && (p - j < a.window || j < a.sinks)));
            if (!see) s[nt][e] = -INFINITY;
          }
      }
      float x0 = fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[1][0], s[1][1]));
      float x1 = fmaxf(fmaxf(s[0][2], s[0][3]), fmaxf(s[1][2], s[1][3]));
#pragma unroll
      for (int d = 1; d < 4; d <<= 1) {
        x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, d));
        x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, d));
      }
      x0 = fmaxf(x0, m0);
      x1 = fmaxf(x1, m1);
      if (__any_sync(0xffffffffu, x0 > m0 || x1 > m1)) {
        const float a0 = ex2(m0 - (x0 == -INFINITY ? 0.f : x0)), a1 = ex2(m1 - (x1 == -INFINITY ? 0.f : x1));
        l0 *= a0;
        l1 *= a1;
#pragma unroll
        for (int i = 0; i < HD / 8; ++i) {
          o[i][0] *= a0;
          o[i][1] *= a0;
          o[i][2] *= a1;
          o[i][3] *= a1;
        }
        m0 = x0;
        m1 = x1;
      }
      const float u0 = m0 == -INFINITY ? 0.f : m0, u1 = m1 == -INFINITY ? 0.f : m1;
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        s[nt][0] = ex2(s[nt][0] - u0);
        s[nt][1] = ex2(s[nt][1] - u0);
        s[nt][2] = ex2(s[nt][2] - u1);
        s[nt][3] = ex2(s[nt][3] - u1);
        l0 += s[nt][0] + s[nt][1];
        l1 += s[nt][2] + s[nt][3];
      }
      const uint32_t pf[4] = {pack2<F16>(s[0][0], s[0][1]), pack2<F16>(s[0][2], s[0][3]),
                              pack2<F16>(s[1][0], s[1][1]), pack2<F16>(s[1][2], s[1][3])};
      {
        const uint32_t base = smem_u32(sv) + ((mi & 1) * 8 + mr) * 128;
#pragma unroll
        for (int nt = 0; nt < HD / 16; ++nt) {
          uint32_t vf[4];
          const int ch = nt * 2 + (mi >> 1);
          ldsm_x4_t(vf, base + (ch >> 3) * 2048 + (((ch & 7) ^ mr) << 4));
          mma<F16>(o[2 * nt], pf, vf[0], vf[1]);
          mma<F16>(o[2 * nt + 1], pf, vf[2], vf[3]);
        }
      }
    }
    __syncwarp();
    if (ok && lane == 0 && u + NST * W < units) issue(u + NST * W, st);
    if (++st == NST) {
      st = 0;
      ph ^= 1;
    }
  }
  if (!ok) l0 = l1 = NAN;  // a copy did not arrive (reported): no result

  // The warps' states meet in shared memory (each in its own ring, drained).
#pragma unroll
  for (int d = 1; d < 4; d <<= 1) {
    l0 += __shfl_xor_sync(0xffffffffu, l0, d);
    l1 += __shfl_xor_sync(0xffffffffu, l1, d);
  }
  __syncwarp();
  float* so = reinterpret_cast<float*>(ring);  // [kRows][HD]
#pragma unroll
  for (int i = 0; i < HD / 8; ++i) {
    *reinterpret_cast<float2*>(so + g * HD + i * 8 + c2) = make_float2(o[i][0], o[i][1]);
    *reinterpret_cast<float2*>(so + (g + 8) * HD + i * 8 + c2) = make_float2(o[i][2], o[i][3]);
  }
  if ((lane & 3) == 0) {
    s_m[warp][g] = m0;
    s_m[warp][g + 8] = m1;
    s_l[warp][g] = l0;
    s_l[warp][g + 8] = l1;
  }
  __syncthreads();
  const int nrow = min(kRows, a.Tq * t.rep - t.row0);
  // the CTA's state per row, in warp 0's ring: one row a warp, lane has dims 2 lane + 64 i
  auto weight = [](float m, float top) { return m == -INFINITY ? 0.f : ex2(m - top); };
  for (int r = warp; r < nrow; r += kWarps) {
    float top = -INFINITY, l = 0.f;
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_m[w][r]);
    float2 acc[HD / 64];
#pragma unroll
    for (int i = 0; i < HD / 64; ++i) acc[i] = make_float2(0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = weight(s_m[w][r], top);
      // a state without keys has l 0 (NaN only after a failed wait: kept)
      l += s_m[w][r] == -INFINITY ? s_l[w][r] : f * s_l[w][r];
      const float* src = reinterpret_cast<const float*>(smem + w * NST * SB) + r * HD + 2 * lane;
      if (f != 0.f) {
#pragma unroll
        for (int i = 0; i < HD / 64; ++i) {
          const float2 v = *reinterpret_cast<const float2*>(src + 64 * i);
          acc[i].x += f * v.x;
          acc[i].y += f * v.y;
        }
      }
    }
    if (sh.apart) {  // (one CTA a tile) to the workspace, as the prefix's parts lie there
      const int i = t.row0 + r, pi = t.b * t.rep + i, rows = a.B * t.rep, pq = pi & 255;
      const PrefixWs ws = prefix_ws(a.ws, pi >> 8, (rows + 255) / 256, rows, t.hk, a.Hkv, presplit, presplit + 1, HD);
#pragma unroll
      for (int i2 = 0; i2 < HD / 64; ++i2) {
        const int d = 2 * lane + 64 * i2;
        *reinterpret_cast<float2*>(ws.o + pq * HD + ((d >> 2) ^ (pq & (HD / 4 - 1))) * 4 + (d & 3)) = acc[i2];
      }
      if (lane == 0) {
        ws.m[pq] = top;
        ws.l[pq] = l;
      }
      continue;
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < HD / 64; ++i)
      *reinterpret_cast<float2*>(reinterpret_cast<float*>(smem) + r * HD + 2 * lane + 64 * i) = acc[i];
    if (lane == 0) {
      c_m[r] = top;
      c_l[r] = l;
    }
  }
  if (sh.apart) {
    // the join follows this kernel: it is not complete before the prefix's is
    if (blockIdx.x == gridDim.x - 1) pdl_wait();
    return;
  }
  if (split > 1)
    cluster_barrier();
  else
    __syncthreads();
  if (a.P > 0) pdl_wait();  // the prefix's part of the rows is complete and visible
  for (int r = part * kWarps + warp; r < nrow; r += W) {
    const int i = t.row0 + r, tq = sh.by_rep.quot(i), gh = i - tq * t.rep, h = t.hk * t.rep + gh;
    if (tq >= t.ql) continue;
    float cm = -INFINITY, cl = 0.f, pm = -INFINITY, pl = 0.f;
    if (lane < split) {
      cm = cluster_ld(cluster_addr(&c_m[r], lane));
      cl = cluster_ld(cluster_addr(&c_l[r], lane));
    }
    PrefixWs ws;
    int pq = 0;
    if (a.P > 0) {
      const int pi = t.b * t.rep + gh, ptiles = (a.B * t.rep + 255) / 256;
      pq = pi & 255;
      ws = prefix_ws(a.ws, pi >> 8, ptiles, a.B * t.rep, t.hk, a.Hkv, 0, presplit, HD);
      if (lane < presplit) {
        const long long at = (long long)lane * 2 * prefix_rows(ptiles, a.B * t.rep) + pq;
        pm = ws.m[at];
        pl = ws.l[at];
      }
    }
    const float top = warp_max(fmaxf(cm, pm));
    const float f = weight(cm, top), fp = weight(pm, top);
    const float l = warp_sum((cm == -INFINITY ? cl : f * cl) + (pm == -INFINITY ? pl : fp * pl));
    float2 acc[HD / 64];
#pragma unroll
    for (int i2 = 0; i2 < HD / 64; ++i2) acc[i2] = make_float2(0.f, 0.f);
    if (a.P > 0) {
      const long long step = (long long)prefix_rows((a.B * t.rep + 255) / 256, a.B * t.rep) * HD;
      const float* src = ws.o + pq * HD + (((2 * lane) >> 2) ^ (pq & (HD / 4 - 1) & 15)) * 4 + (2 * lane & 3);
      for (int c0 = 0; c0 < presplit; c0 += 8) {  // eight parts' loads in flight together
        float2 v[8][HD / 64];
#pragma unroll
        for (int c = 0; c < 8; ++c)
#pragma unroll
          for (int i2 = 0; i2 < HD / 64; ++i2)
            v[c][i2] = *reinterpret_cast<const float2*>(src + min(c0 + c, presplit - 1) * step +
                                                        (HD == 128 ? 64 * (i2 ^ ((pq >> 4) & 1)) : 0));
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const float fc = __shfl_sync(0xffffffffu, fp, (c0 + c) & 31);
          if (c0 + c >= presplit || fc == 0.f) continue;
#pragma unroll
          for (int i2 = 0; i2 < HD / 64; ++i2) {
            acc[i2].x += fc * v[c][i2].x;
            acc[i2].y += fc * v[c][i2].y;
          }
        }
      }
    }
    const uint32_t own = smem_u32(reinterpret_cast<float*>(smem) + r * HD + 2 * lane);
    for (int c0 = 0; c0 < split; c0 += 4) {  // four CTAs' loads in flight together
      float2 v[4][HD / 64];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint32_t src = cluster_map(own, min(c0 + c, split - 1));
#pragma unroll
        for (int i2 = 0; i2 < HD / 64; ++i2) v[c][i2] = cluster_ld2(src + 256 * i2);
      }
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float fc = __shfl_sync(0xffffffffu, f, c0 + c);
        if (c0 + c >= split || fc == 0.f) continue;
#pragma unroll
        for (int i2 = 0; i2 < HD / 64; ++i2) {
          acc[i2].x += fc * v[c][i2].x;
          acc[i2].y += fc * v[c][i2].y;
        }
      }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    bool fin = true;
    const long long at = t.b * a.os[0] + tq * a.os[1] + h * a.os[2] + 2 * lane;
#pragma unroll
    for (int i2 = 0; i2 < HD / 64; ++i2) {
      const float x = acc[i2].x * inv, y = acc[i2].y * inv;
      fin = fin && isfinite(x) && isfinite(y);
      *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + at + 64 * i2) = pack2<F16>(x, y);
    }
    if (lane == 0 && a.lse)
      a.lse[((long long)t.b * a.Tq + tq) * a.Hq + h] = l == 0.f ? -INFINITY : (top + log2f(l)) * 0.6931471805599453f;
    // rows of different masks shared this tile's V rows: a row that is not
    // finite may owe that to a key it does not see (0 * infinity)
    if (!one_mask && !__all_sync(0xffffffffu, fin) && ok) exact_row<HD, F16>(a, t.b, tq, h, t.n, t.ql, lane);
  }
  if (split > 1) cluster_barrier();  // nobody leaves while its shared memory may still be read
}

// A warp a row: the parts' maxima and sums a lane each, their outputs eight at a
// time; as above.
template <int HD, bool F16>
__global__ void __launch_bounds__(256) k_prefix_join(const __grid_constant__ AttnOpArgs a, int parts, FastDiv by_rows, FastDiv by_rep) {
  const int lane = threadIdx.x & 31, id = blockIdx.x * 8 + (threadIdx.x >> 5), rows = by_rows.d;
  const int hk = by_rows.quot(id), pi = id - hk * rows;
  if (hk >= a.Hkv) return;
  const int b = by_rep.quot(pi), h = hk * by_rep.d + pi - b * by_rep.d, pq = pi & 255, ptiles = (rows + 255) / 256;
  const PrefixWs ws = prefix_ws(a.ws, pi >> 8, ptiles, rows, hk, a.Hkv, 0, parts, HD);
  const long long R = prefix_rows(ptiles, rows);
  float pm = -INFINITY, pl = 0.f;
  if (lane < parts) {
    pm = ws.m[lane * 2 * R + pq];
    pl = ws.l[lane * 2 * R + pq];
  }
  const float top = warp_max(pm), f = pm == -INFINITY ? 0.f : ex2(pm - top);
  const float l = warp_sum(pm == -INFINITY ? pl : f * pl);
  float2 acc[HD / 64];
#pragma unroll
  for (int i = 0; i < HD / 64; ++i) acc[i] = make_float2(0.f, 0.f);
  for (int c0 = 0; c0 < parts; c0 += 8) {
    float2 v[8][HD / 64];
#pragma unroll
    for (int c = 0; c < 8; ++c)
#pragma unroll
      for (int i = 0; i < HD / 64; ++i) {
        const int d = 2 * lane + 64 * i;
        v[c][i] = *reinterpret_cast<const float2*>(ws.o + min(c0 + c, parts - 1) * R * HD + pq * HD +
                                                   ((d >> 2) ^ (pq & (HD / 4 - 1))) * 4 + (d & 3));
      }
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const float fc = __shfl_sync(0xffffffffu, f, (c0 + c) & 31);
      if (c0 + c >= parts || fc == 0.f) continue;
#pragma unroll
      for (int i = 0; i < HD / 64; ++i) {
        acc[i].x += fc * v[c][i].x;
        acc[i].y += fc * v[c][i].y;
      }
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int i = 0; i < HD / 64; ++i)
    *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + b * a.os[0] + h * a.os[2] + 2 * lane + 64 * i) =
        pack2<F16>(acc[i].x * inv, acc[i].y * inv);
  if (lane == 0 && a.lse) a.lse[(long long)b * a.Hq + h] = l == 0.f ? -INFINITY : (top + log2f(l)) * 0.6931471805599453f;
}

// CTAs a row tile's keys are split over: as many as keep all of them within two
// a SM, a unit for each warp.  More only queue clusters behind one another:
// head_dim 128, window 2048, 8 KV heads: one sequence 26.3 us in 1 part, 11.9 in
// 4, 9.3 in 8, 8.1 in 12, 9.3 in 16; 8 sequences 27.1, 16.4, 24.4, 23.1, 37.0;
// 32 sequences 43.8 us in 1 part, 54.8 in 4.
int pick_split(long long tiles, int keys, int sm_count) {
  const int units = (keys + kUnit - 1) / kUnit;
  const long long s = min(2ll * sm_count / tiles, (long long)(units + kWarps - 1) / kWarps);
  return (int)max(1ll, min(s, (long long)kMaxSplit));
}

template <int HD, bool F16>
cudaError_t launch(const AttnOpArgs& a, bool pdl, cudaStream_t s) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = device_sm_count(dev, &sms);
  if (e != cudaSuccess) return e;
  auto kern = k_attn_decode<HD, F16>;
  {
    static std::mutex mu;
    static bool done[kOpDevices] = {};
    std::lock_guard<std::mutex> lock(mu);
    if (!done[dev]) {
      e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem<HD>);
      if (e == cudaSuccess) e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
      if (e != cudaSuccess) return e;
      done[dev] = true;
    }
  }
  KvMaps maps;
  if (!make_kv_maps(&maps, a.kv, a.f16 != 0, a.B, a.Hkv, HD, a.cap, kUnit)) return cudaErrorInvalidValue;
  const int tiles = (a.Tq * (a.Hq / a.Hkv) + kRows - 1) / kRows;
  const long long all = (long long)a.B * a.Hkv * tiles;
  const int presplit = a.P > 0 ? prefix_split(a.B, a.Hq / a.Hkv, a.Hkv, a.P) : 0;
  const int apart = a.P > 0 && prefix_apart(a.B, a.Hq / a.Hkv, a.Hkv);
  const int split = apart ? 1 : pick_split(all, (int)min((long long)a.cap, (long long)a.window + a.Tq + a.sinks), sms);
  if (all * split >= (1ll << 31)) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(all * split));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem<HD>;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = split;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 2 : 1;
  const DecodeShape sh{split, tiles, presplit, apart, FastDiv(split), FastDiv(tiles), FastDiv(a.Hkv), FastDiv(a.Hq / a.Hkv)};
  return cudaLaunchKernelEx(&cfg, kern, maps, a, sh);
}

}  // namespace

namespace attn {

bool make_kv_maps(KvMaps* m, const KeySrc& s, bool f16, int B, int Hkv, int hd, int tokens, int rows) {
  const PFN_cuTensorMapEncodeTiled_v12000 fn = tensor_map_encoder();
  if (fn == nullptr) return false;
  const CUtensorMapDataType dt = f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  auto one = [&](CUtensorMap* map, const void* base, const long long (&st)[3], int* seq_mul, int* head_mul) {
    *seq_mul = st[0] != 0;
    *head_mul = st[1] != 0;
    const cuuint64_t dims[5] = {64, (cuuint64_t)tokens, (cuuint64_t)(hd / 64), (cuuint64_t)(st[1] ? Hkv : 1),
                                (cuuint64_t)(st[0] ? B : 1)};
    // (an axis of extent 1 takes any stride)
    const cuuint64_t strides[4] = {(cuuint64_t)(st[2] ? st[2] : hd) * 2, 128, (cuuint64_t)(st[1] ? st[1] : hd) * 2,
                                   (cuuint64_t)(st[0] ? st[0] : hd) * 2};
    const cuuint32_t box[5] = {64, (cuuint32_t)rows, (cuuint32_t)(hd / 64), 1, 1};
    const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
    return fn(map, dt, 5, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  return one(&m->k, s.k, s.ks, &m->kb, &m->kh) && one(&m->v, s.v, s.vs, &m->vb, &m->vh);
}

}  // namespace attn

cudaError_t launch_prefix_join(const AttnOpArgs& a, cudaStream_t s) {
  const int rep = a.Hq / a.Hkv, rows = a.B * rep, parts = prefix_split(a.B, rep, a.Hkv, a.P) + 1;
  const unsigned grid = (unsigned)(((long long)rows * a.Hkv + 7) / 8);
  const FastDiv by_rows(rows), by_rep(rep);
  if (a.hd == 64)
    a.f16 ? k_prefix_join<64, true><<<grid, 256, 0, s>>>(a, parts, by_rows, by_rep)
          : k_prefix_join<64, false><<<grid, 256, 0, s>>>(a, parts, by_rows, by_rep);
  else
    a.f16 ? k_prefix_join<128, true><<<grid, 256, 0, s>>>(a, parts, by_rows, by_rep)
          : k_prefix_join<128, false><<<grid, 256, 0, s>>>(a, parts, by_rows, by_rep);
  return cudaGetLastError();
}

cudaError_t launch_attn_decode(const AttnOpArgs& a, bool pdl, cudaStream_t s) {
  if (a.hd == 64) return a.f16 ? launch<64, true>(a, pdl, s) : launch<64, false>(a, pdl, s);
  return a.f16 ? launch<128, true>(a, pdl, s) : launch<128, false>(a, pdl, s);
}

}  // namespace river
