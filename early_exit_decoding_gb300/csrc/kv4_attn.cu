// Attention over the paged cache held in 4 bits (rl_kv4_attention): single
// tokens and drafts.
//
// A key's value is m + s c with a code c of 4 bits, so for a query row q
//   q.k_j = s_j (q.c_j) + m_j sum(q)
//   sum_j w_j v_j = sum_j (w_j s_j)(c_j - 8) + sum_j w_j (m_j + 8 s_j)
// and the tensor cores multiply codes: a code in the low bits of a half is the
// fp16 number c 2^-24, exact, so a mask (no conversion) turns a word of eight
// codes into operands; the second code of a byte stands for 16 times that,
// which q (for k) or the result's row (for v) takes back.  Codes are the A
// operand of m16n8k16, 16 keys (q.c) or 16 dims (w.c) a tile, and 8 or 16 query
// rows the B operand.  Which dim of a code word meets which k index is free as
// long as q has the same order, so a lane's operands are whole words of its
// own: a 16-byte load of k gives it 32 of a key's dims, 8 bytes of v 16 dims
// of a key.
//
// Numbers: q is scaled by a power of two a row (its largest to 2^13), exact in
// fp16 but for what is 2^-37 below the largest.  The weights times s go to fp16
// relative to the largest of them so far, 2^M, apart from the softmax's own
// maximum m: steps may be of any size.  That rounding (2^-12 of a weight) meets
// c - 8, as the sum of the rounded weights comes from the same products (a row
// of eights beside the codes).  Scores, sums and statistics are fp32.  Maxima
// follow lazily: everything is rescaled only when one grew by more than 2^8.
//
// Each warp runs its own ring: 32 keys a stage, copied by 4 or 8 bulk copies
// (codes and scales of k and v; a page's rows of a head are contiguous).  Keys
// are dealt out unit by unit to the warps of a cluster of S CTAs and the states
// joined at the end, as in attn_decode.cu: no workspace, one launch.
#include <float.h>
#include <math.h>

#include <stdlib.h>
#include <mutex>

#include "kv4.cuh"

namespace river {

namespace {

using namespace dev;
using namespace attn;

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kUnit = 32;      // keys a warp takes at a time
constexpr int kMaxSplit = 16;  // CTAs of a cluster
constexpr unsigned long long kWaitNs = 2000000000ull;  // a wait gives up after two seconds
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLazy = 8.f;   // log2 growth of a maximum that is let pass

template <int HD>
constexpr int kStageBytes = kUnit * HD + 2 * kUnit * 4;  // codes of k and v, scales of k and v
template <int HD>
constexpr int kStages = HD == 128 ? 4 : 8;
template <int HD>
constexpr int kSmem = kWarps * kStages<HD> * kStageBytes<HD>;

struct Kv4Shape {
  int split, tiles;  // CTAs of a cluster; row tiles of a sequence (without start)
  FastDiv by_split, by_heads, by_rep, by_tiles;
};

__device__ __forceinline__ uint32_t transposed(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float pivot(float m) { return m == -INFINITY ? 0.f : m; }

template <int HD, bool F16, int NT>
__global__ void __launch_bounds__(kThreads, 3)
    k_kv4_attn(const __grid_constant__ PackedArgs a, const __grid_constant__ Kv4Args c, const __grid_constant__ Kv4Shape sh) {
  constexpr int NST = kStages<HD>, SB = kStageBytes<HD>, R = 8 * NT, KW = HD / 32;  // KW: words of k's codes a lane takes
  constexpr uint32_t kLow = 0x000f000fu, kHigh = 0x00f000f0u;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ __align__(8) uint64_t full[kWarps][NST];
  __shared__ float s_m[kWarps][R], s_l[kWarps][R];
  __shared__ float c_m[R], c_l[R];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  check_start(a);
  const int id = sh.by_split.quot(blockIdx.x), part = blockIdx.x - id * sh.split;
  const int tile = sh.by_heads.quot(id), hk = id - tile * sh.by_heads.d, rep = sh.by_rep.d;
  int b, row0;
  if (a.start) {
    RowTile rt;
    if (!row_tile(a.start, a.B, a.N, a.max_rows, rep, R, tile, lane, &rt)) return;  // (its whole cluster)
    b = rt.seq;
    row0 = rt.number * R;
  } else {
    b = sh.by_tiles.quot(tile);
    row0 = (tile - b * sh.tiles) * R;
  }
  const bool report = part == 0 && hk == 0 && row0 == 0 && tid == 0;
  const Span sp = seq_span(a, b, report);
  const int cap = c.width << c.page_log, len = __ldg(a.kv_len + b);
  if (report && a.err && (len < 0 || len > cap)) atomicOr(a.err, RL_DEVERR_CAPACITY);
  const int old = max(0, min(len, cap)) - sp.all;  // position of the sequence's first row here
  const int nrow = min(R, sp.n * rep - row0);
  if (nrow <= 0) return;
  // keys that every row sees, and that any row sees
  const int every = old + sh.by_rep.quot(row0) + 1, any = max(0, old + sh.by_rep.quot(row0 + nrow - 1) + 1);
  const int units = (any + kUnit - 1) / kUnit, W = sh.split * kWarps, first = part * kWarps + warp;

  unsigned char* ring = smem + warp * NST * SB;
  if (lane == 0) {
    for (int i = 0; i < NST; ++i) mbar_init(&full[warp][i], 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncwarp();
  // lanes 0-7 copy: 16 keys (lane / 4) of k's codes, k's scales, v's codes, v's
  // scales (lane % 4); where a page holds a whole unit lanes 0-3 all of it
  const int sub = (lane >> 2) & 1, what = lane & 3;
  auto page_of = [&](int u) {  // page of this lane's keys of unit u
    const int j = u * kUnit + sub * 16;
    return lane < 8 && j < any ? max(0, page_at(a, c, b, j >> c.page_log)) : 0;
  };
  auto issue = [&](int u, int st, int page) {
    unsigned char* dst = ring + st * SB;
    const int nsub = any - u * kUnit > 16 ? 2 : 1;
    const bool whole = nsub == 2 && c.page_log >= 5;
    if (lane == 0) mbar_expect_tx(&full[warp][st], nsub * (16 * HD + 128));
    __syncwarp();
    if (lane < (whole ? 4 : 4 * nsub)) {
      const long long at = page_row(c, hk, (u * kUnit + sub * 16) & ((1 << c.page_log) - 1));
      const int n = whole ? kUnit : 16;
      const unsigned char* src;
      if (what == 0)
        src = c.kc + page * c.kc_step + at * (HD / 2);
      else if (what == 1)
        src = reinterpret_cast<const unsigned char*>(c.km + page * c.km_step + at);
      else if (what == 2)
        src = c.vc + page * c.vc_step + at * (HD / 2);
      else
        src = reinterpret_cast<const unsigned char*>(c.vm + page * c.vm_step + at);
      const int row = what & 1 ? 4 : HD / 2;
      // stage: k's codes, v's codes, k's scales, v's scales
      dst += (what == 0 ? 0 : what == 2 ? kUnit * HD / 2 : what == 1 ? kUnit * HD : kUnit * HD + kUnit * 4) + sub * 16 * row;
      bulk_g2s(dst, src, n * row, &full[warp][st]);
    }
  };
#pragma unroll
  for (int i = 0; i < NST; ++i)
    if (first + i * W < units) issue(first + i * W, i, page_of(first + i * W));

  // B operands of q: this lane has row g of each tile, dims 32 t (16 t) and on
  uint32_t qb[NT][2 * KW][2];
  float mul[NT][2], qsum[NT][2];  // of the rows 2 t and 2 t + 1: scores are acc mul s + qsum m
  int end[NT][2];                 // and the keys they see
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int i = row0 + nt * 8 + g, tq = sh.by_rep.quot(i);
    float2 f[4 * KW];
    float big = 0.f, sum = 0.f;
    const bool live = nt * 8 + g < nrow;
    const uint16_t* src = static_cast<const uint16_t*>(a.q) + (long long)(sp.first + (live ? tq : 0)) * a.qs[0] +
                          (long long)(hk * rep + (live ? i - tq * rep : 0)) * a.qs[1] + 8 * KW * t;
#pragma unroll
    for (int w = 0; w < KW; ++w) {
      const uint4 x = *reinterpret_cast<const uint4*>(src + 8 * w);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 v = unpack2<F16>(live ? u4get(x, e) : 0u);
        f[4 * w + e] = v;
        big = fmaxf(big, fmaxf(fabsf(v.x), fabsf(v.y)));
        sum += v.x + v.y;
      }
    }
#pragma unroll
    for (int d = 1; d < 4; d <<= 1) {
      big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, d));
      sum += __shfl_xor_sync(0xffffffffu, sum, d);
    }
    // 2^e <= the largest < 2^(e + 1); rows of zeros and below 2^-100 as if it were 2^-100
    const int e = max((int)((__float_as_uint(big) >> 23) & 255) - 127, -100);
    const float up = __uint_as_float((uint32_t)(127 + min(13 - e, 127)) << 23), up16 = up * 0.0625f;
#pragma unroll
    for (int w = 0; w < KW; ++w) {
      const float2* v = f + 4 * w;  // dims 0 1, 2 3, 4 5, 6 7 of the word
      qb[nt][2 * w][0] = pack2<true>(v[0].x * up, v[2].x * up);
      qb[nt][2 * w][1] = pack2<true>(v[0].y * up16, v[2].y * up16);
      qb[nt][2 * w + 1][0] = pack2<true>(v[1].x * up, v[3].x * up);
      qb[nt][2 * w + 1][1] = pack2<true>(v[1].y * up16, v[3].y * up16);
    }
    const float sc = a.scale * kLog2e, back = sc * 16777216.f / up;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      mul[nt][r] = __shfl_sync(0xffffffffu, back, (2 * t + r) * 4);
      qsum[nt][r] = __shfl_sync(0xffffffffu, sum * sc, (2 * t + r) * 4);
      end[nt][r] = old + sh.by_rep.quot(row0 + nt * 8 + 2 * t + r) + 1;
    }
  }

  float o[NT][HD / 16][4], o8[NT][4];  // sums over codes: dims (rows) g and g + 8 of a tile, query rows 2 t, 2 t + 1
  float m[NT][2], M[NT][2], l[NT][2], z[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int i = 0; i < HD / 16; ++i) o[nt][i][0] = o[nt][i][1] = o[nt][i][2] = o[nt][i][3] = 0.f;
    o8[nt][0] = o8[nt][1] = o8[nt][2] = o8[nt][3] = 0.f;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      m[nt][r] = M[nt][r] = -INFINITY;
      l[nt][r] = z[nt][r] = 0.f;
    }
  }
  // Key of a tile's row g: neighbours swapped in every second pair, so that the
  // loads of k (rows g, lanes t) and of v (rows 2 t, 2 t + 1, lanes g) both
  // spread over the banks.
  const int kg = g ^ ((g >> 1) & 1), ka = (2 * t) ^ (t & 1), kb = ka ^ 1;
  int st = 0, ph = 0, stop = units;
  bool ok = true;
  int next = first + NST * W < units ? page_of(first + NST * W) : 0;  // page of the unit to be copied next
  // After a wait that gave up nothing is copied or computed any more; the
  // copies already in flight are still waited for (`stop`).
  for (int u = first; u < stop; u += W) {
    const bool got = mbar_wait_lazy(&full[warp][st], ph, kWaitNs);
    if (!__all_sync(0xffffffffu, got) && ok) {
      ok = false;
      stop = min(units, u + NST * W);
      if (lane == 0 && a.err) atomicOr(a.err, RL_DEVERR_TIMEOUT);
    }
    if (ok) {
      const unsigned char* sk = ring + st * SB;
      const unsigned char* sv = sk + kUnit * HD / 2;
      const uint32_t* sm = reinterpret_cast<const uint32_t*>(sk + kUnit * HD);
      const int j0 = u * kUnit;
      const bool cut = j0 + kUnit > every;
      float s[2][NT][4], tv[2][NT][4], vm8[2][2];  // scores; plus log2 of v's step; v's m + 8 s of keys g, g + 8
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        uint32_t w[2][KW];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const unsigned char* src = sk + (q * 16 + h * 8 + kg) * (HD / 2) + t * (HD / 8);
          if constexpr (HD == 128) {
            const uint4 x = *reinterpret_cast<const uint4*>(src);
            w[h][0] = x.x;
            w[h][1] = x.y;
            w[h][2] = x.z;
            w[h][3] = x.w;
          } else {
            const uint2 x = *reinterpret_cast<const uint2*>(src);
            w[h][0] = x.x;
            w[h][1] = x.y;
          }
        }
        float acc[NT][4] = {};
#pragma unroll
        for (int i = 0; i < KW; ++i) {
          const uint32_t x0 = w[0][i] >> 8, x1 = w[1][i] >> 8;
          const uint32_t lo[4] = {w[0][i] & kLow, w[1][i] & kLow, w[0][i] & kHigh, w[1][i] & kHigh};
          const uint32_t hi[4] = {x0 & kLow, x1 & kLow, x0 & kHigh, x1 & kHigh};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma_f16(acc[nt], lo[0], lo[1], lo[2], lo[3], qb[nt][2 * i][0], qb[nt][2 * i][1]);
            mma_f16(acc[nt], hi[0], hi[1], hi[2], hi[3], qb[nt][2 * i + 1][0], qb[nt][2 * i + 1][1]);
          }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int key = q * 16 + h * 8 + kg;
          const float2 km = unpack2<F16>(sm[key]), vm = unpack2<F16>(sm[kUnit + key]);
          const float lv = lg2(vm.x);
          vm8[q][h] = fmaf(8.f, vm.x, vm.y);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const float x = fmaf(acc[nt][2 * h + r] * mul[nt][r], km.x, km.y * qsum[nt][r]);
              s[q][nt][2 * h + r] = x;
              tv[q][nt][2 * h + r] = x + lv;
            }
        }
      }
      if (cut) {
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (j0 + q * 16 + (e >> 1) * 8 + kg >= end[nt][e & 1]) s[q][nt][e] = tv[q][nt][e] = -INFINITY;
      }
      float x[NT][2], y[NT][2];
      bool up = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          x[nt][r] = fmaxf(fmaxf(s[0][nt][r], s[0][nt][2 + r]), fmaxf(s[1][nt][r], s[1][nt][2 + r]));
          y[nt][r] = fmaxf(fmaxf(tv[0][nt][r], tv[0][nt][2 + r]), fmaxf(tv[1][nt][r], tv[1][nt][2 + r]));
          up = up || x[nt][r] > m[nt][r] + kLazy || y[nt][r] > M[nt][r] + kLazy;
        }
      if (__any_sync(0xffffffffu, up)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float fo[2];
#pragma unroll
          for (int r = 0; r < 2; ++r) {
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) {
              x[nt][r] = fmaxf(x[nt][r], __shfl_xor_sync(0xffffffffu, x[nt][r], d));
              y[nt][r] = fmaxf(y[nt][r], __shfl_xor_sync(0xffffffffu, y[nt][r], d));
            }
            const float mn = fmaxf(m[nt][r], x[nt][r]), Mn = fmaxf(M[nt][r], y[nt][r]);
            const float f = ex2(m[nt][r] - pivot(mn));
            fo[r] = ex2(M[nt][r] - pivot(Mn));
            m[nt][r] = mn;
            M[nt][r] = Mn;
            l[nt][r] *= f;
            z[nt][r] *= f;
          }
#pragma unroll
          for (int i = 0; i < HD / 16; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[nt][i][e] *= fo[e & 1];
#pragma unroll
          for (int e = 0; e < 4; ++e) o8[nt][e] *= fo[e & 1];
        }
      }
      uint32_t p[2][NT][2];  // B operands: weights times steps
#pragma unroll
      for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float e[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float w = ex2(s[q][nt][i] - pivot(m[nt][i & 1]));
            l[nt][i & 1] += w;
            // (a key that a row does not see may hold anything)
            z[nt][i & 1] = fmaf(w, cut && s[q][nt][i] == -INFINITY ? 0.f : vm8[q][i >> 1], z[nt][i & 1]);
            e[i] = ex2(tv[q][nt][i] - pivot(M[nt][i & 1]));
          }
          p[q][nt][0] = transposed(pack2<true>(e[0], e[1]));
          p[q][nt][1] = transposed(pack2<true>(e[2], e[3]));
        }
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        uint32_t w[4][HD / 64];  // codes of four keys: this lane's dims
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          const unsigned char* src = sv + (q * 16 + (h >> 1) * 8 + (h & 1 ? kb : ka)) * (HD / 2) + g * (HD / 16);
          if constexpr (HD == 128) {
            const uint2 x = *reinterpret_cast<const uint2*>(src);
            w[h][0] = x.x;
            w[h][1] = x.y;
          } else {
            w[h][0] = *reinterpret_cast<const uint32_t*>(src);
          }
        }
#pragma unroll
        for (int i = 0; i < HD / 64; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h) {  // dims 0-3, 4-7 of the word: of keys a b, and of keys c d
            const uint32_t x = __byte_perm(w[0][i], w[1][i], h ? 0x7632 : 0x5410), y = __byte_perm(w[2][i], w[3][i], h ? 0x7632 : 0x5410);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const uint32_t xx = e ? x >> 8 : x, yy = e ? y >> 8 : y;
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma_f16(o[nt][4 * i + 2 * h + e], xx & kLow, xx & kHigh, yy & kLow, yy & kHigh, p[q][nt][0], p[q][nt][1]);
            }
          }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          mma_f16(o8[nt], 0x00080008u, 0x00080008u, 0x00080008u, 0x00080008u, p[q][nt][0], p[q][nt][1]);
      }
    }
    __syncwarp();
    if (ok && u + NST * W < units) {
      issue(u + NST * W, st, next);
      if (u + (NST + 1) * W < units) next = page_of(u + (NST + 1) * W);
    }
    if (++st == NST) {
      st = 0;
      ph ^= 1;
    }
  }

  // The warps' states meet in shared memory (each in its own ring, drained):
  // sums of weighted values, as [R][HD].
  __syncwarp();
  float* so = reinterpret_cast<float*>(ring);
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) {
        l[nt][r] += __shfl_xor_sync(0xffffffffu, l[nt][r], d);
        z[nt][r] += __shfl_xor_sync(0xffffffffu, z[nt][r], d);
      }
      if (!ok) l[nt][r] = NAN;  // a copy did not arrive (reported): no result
      const float f = M[nt][r] == -INFINITY ? 0.f : ex2(M[nt][r] - m[nt][r] + 20.f);
      const int row = nt * 8 + 2 * t + r;
#pragma unroll
      for (int i = 0; i < HD / 16; ++i) {
        const float even = (o[nt][i][r] - o8[nt][r]) * 16.f, odd = o[nt][i][2 + r] - 16.f * o8[nt][r];
        *reinterpret_cast<float2*>(so + row * HD + g * (HD / 8) + 2 * i) = make_float2(fmaf(even, f, z[nt][r]), fmaf(odd, f, z[nt][r]));
      }
      if (g == 0) {
        s_m[warp][row] = m[nt][r];
        s_l[warp][row] = l[nt][r];
      }
    }
  __syncthreads();
  // the CTA's state per row, in warp 0's ring: one row a warp, lane has dims 2 lane + 64 i
  auto weight = [](float x, float top) { return x == -INFINITY ? 0.f : ex2(x - top); };
  for (int r = warp; r < nrow; r += kWarps) {
    float top = -INFINITY, sum = 0.f;
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_m[w][r]);
    float2 acc[HD / 64];
#pragma unroll
    for (int i = 0; i < HD / 64; ++i) acc[i] = make_float2(0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = weight(s_m[w][r], top);
      // a state without keys has sum 0 (NaN only after a failed wait, or of NaN scores: kept)
      sum += s_m[w][r] == -INFINITY ? s_l[w][r] : f * s_l[w][r];
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
    __syncwarp();
#pragma unroll
    for (int i = 0; i < HD / 64; ++i) *reinterpret_cast<float2*>(reinterpret_cast<float*>(smem) + r * HD + 2 * lane + 64 * i) = acc[i];
    if (lane == 0) {
      c_m[r] = top;
      c_l[r] = sum;
    }
  }
  if (sh.split > 1)
    cluster_barrier();
  else
    __syncthreads();
  for (int r = part * kWarps + warp; r < nrow; r += W) {
    const int i = row0 + r, tq = sh.by_rep.quot(i), h = hk * rep + i - tq * rep;
    float cm = -INFINITY, cl = 0.f;
    if (lane < sh.split) {
      cm = cluster_ld(cluster_addr(&c_m[r], lane));
      cl = cluster_ld(cluster_addr(&c_l[r], lane));
    }
    const float top = warp_max(cm), f = weight(cm, top), sum = warp_sum(cm == -INFINITY ? cl : f * cl);
    float2 acc[HD / 64];
#pragma unroll
    for (int i2 = 0; i2 < HD / 64; ++i2) acc[i2] = make_float2(0.f, 0.f);
    const uint32_t own = smem_u32(reinterpret_cast<float*>(smem) + r * HD + 2 * lane);
    for (int c0 = 0; c0 < sh.split; c0 += 4) {  // four CTAs' loads in flight together
      float2 v[4][HD / 64];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t src = cluster_map(own, min(c0 + q, sh.split - 1));
#pragma unroll
        for (int i2 = 0; i2 < HD / 64; ++i2) v[q][i2] = cluster_ld2(src + 256 * i2);
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float fq = __shfl_sync(0xffffffffu, f, (c0 + q) & 31);
        if (c0 + q >= sh.split || fq == 0.f) continue;
#pragma unroll
        for (int i2 = 0; i2 < HD / 64; ++i2) {
          acc[i2].x += fq * v[q][i2].x;
          acc[i2].y += fq * v[q][i2].y;
        }
      }
    }
    // (sum NaN: of a visible key's NaN, or a failed wait)
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const long long at = (long long)(sp.first + tq) * a.os[0] + (long long)h * a.os[1] + 2 * lane;
#pragma unroll
    for (int i2 = 0; i2 < HD / 64; ++i2)
      *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + at + 64 * i2) = pack2<F16>(acc[i2].x * inv, acc[i2].y * inv);
    if (lane == 0 && a.lse)
      a.lse[(long long)(sp.first + tq) * a.Hq + h] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
  }
  if (sh.split > 1) cluster_barrier();  // nobody leaves while its shared memory may still be read
}

template <int HD, bool F16, int NT>
cudaError_t launch(const PackedArgs& p, const Kv4Args& c, cudaStream_t s) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = device_sm_count(dev, &sms);
  if (e != cudaSuccess) return e;
  auto kern = k_kv4_attn<HD, F16, NT>;
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
  const int rep = p.Hq / p.Hkv, most = p.start ? p.max_rows : 1;
  const long long each = ((long long)most * rep + 8 * NT - 1) / (8 * NT);
  const long long tiles = p.start ? min(each * p.B, (long long)p.N * rep / (8 * NT) + p.B) : each * p.B;
  const long long items = tiles * p.Hkv;
  const long long units = (((long long)c.width << c.page_log) + kUnit - 1) / kUnit;
  int split = (int)max(1ll, min(min(4ll * 3 * sms / items, (units + kWarps - 1) / kWarps), (long long)kMaxSplit));
  if (const char* x = getenv("RL_SPLIT")) split = atoi(x);
  if (each >= 1ll << 31 || items * split >= 1ll << 31) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(items * split));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem<HD>;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = split;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const Kv4Shape sh{split, (int)each, FastDiv(split), FastDiv(p.Hkv), FastDiv(rep), FastDiv((int)each)};
  return cudaLaunchKernelEx(&cfg, kern, p, c, sh);
}

template <int HD, bool F16>
cudaError_t launch_rows(const PackedArgs& p, const Kv4Args& c, cudaStream_t s) {
  const long long rows = (long long)(p.start ? p.max_rows : 1) * (p.Hq / p.Hkv);
  return rows <= 8 ? launch<HD, F16, 1>(p, c, s) : launch<HD, F16, 2>(p, c, s);
}

}  // namespace

cudaError_t launch_kv4_attention(const PackedArgs& p, const Kv4Args& c, cudaStream_t s) {
  if (p.hd == 64) return p.f16 ? launch_rows<64, true>(p, c, s) : launch_rows<64, false>(p, c, s);
  return p.f16 ? launch_rows<128, true>(p, c, s) : launch_rows<128, false>(p, c, s);
}

}  // namespace river

using namespace river;

extern "C" rl_status rl_kv4_attention(const rl_kv4* c, const rl_packed_desc* p, const int32_t* d_start, const int32_t* d_kv_len,
                                      const void* d_q, void* d_out, float* d_lse, int32_t* d_err, rl_stream_t stream) {
  const char* who = "rl_kv4_attention";
  PackedArgs a;
  Kv4Args k;
  rl_status st = check_packed(who, p, kUsesQ, kUsesOut, &a);
  if (st == RL_OK) st = check_kv4(who, c, a, &k);
  if (st != RL_OK) return st;
  if (!d_kv_len || !d_q || !d_out || d_out == d_q) return op_error(who, RL_ERR_INVALID_ARG, "NULL argument, or out in q's place");
  if (!d_start && p->rows != p->batch) return op_error(who, RL_ERR_INVALID_ARG, "rows must be batch without d_start");
  if (!op_aligned16(d_q) || !op_aligned16(d_out)) return op_error(who, RL_ERR_UNSUPPORTED, "q and out must start on 16-byte boundaries");
  a.q = d_q;
  a.out = d_out;
  a.lse = d_lse;
  a.start = d_start;
  a.kv_len = d_kv_len;
  a.err = d_err;
  const cudaError_t e = launch_kv4_attention(a, k, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return set_error(RL_ERR_CUDA, cudaGetErrorString(e));
  return RL_OK;
}
