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
// Numbers: q is scaled by a power of two a row (its largest to 2^13, for odd dims,
// whose codes stand for 16 times theirs, to 2^9), exact in fp16 but for what is
// 2^-37 (odd dims: 2^-33) below the largest.  The weights times s go to fp16
// relative to the largest of them so far, 2^M, apart from the softmax's own
// maximum m: steps may be of any size and sign, 0 among them (M is at least
// m - 100, so that it has a value while all steps so far are 0).  That rounding
// (2^-12 of a weight) meets c - 8, as the sum of the rounded weights comes from
// the same products (a row of eights beside the codes); weights times steps
// below 2^-25 of the largest have no part in it.  Scores, sums and statistics are fp32.  Maxima
// follow lazily: everything is rescaled only when one grew by more than 2^8.
//
// Work is counted in units of 32 keys of a row tile and KV head, over the whole
// batch, and each CTA takes an equal, contiguous share of it, however ragged the
// contexts are: the end of one sequence, whole ones, the start of another.  A
// tile whose keys fall to one CTA is finished there; the others' states (sums of
// weighted values, maximum, sum of weights) go to the workspace, at most two a
// CTA, and a second kernel joins them in a fixed order.  Within a share the
// warps take the units in turn, each with a ring of its own filled by
// asynchronous copies.
//
// What bounds it: the chain inside a warp, with three warps a scheduler.  A unit
// of 32 keys of head_dim 128 is 4352 bytes (186 clocks of an SM's share of HBM)
// and takes 34 products and some 520 instructions a warp one after another:
// loads from shared memory, masks (220 with shifts and permutes, on a pipe that
// takes two clocks each), products, exponentials, products.  No unit is at its
// peak: issue slots 52 %, that pipe 51 %, tensor pipe 27 %, DRAM 0.71 of a
// measured copy within the kernel.  64 sequences of 130 to 8191 positions, 8 KV
// heads: 69 us for 291 MB, 4.2 TB/s (0.63 of a copy); two of 99,999 and 131,072:
// 58 us, 4.4 TB/s.  One sequence of 1001: 9.5 us and 6 for the join, latencies.
#include <float.h>
#include <math.h>

#include <mutex>

#include "kv4.cuh"

namespace river {

namespace {

using namespace dev;
using namespace attn;

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kUnit = 32;       // keys a warp takes at a time
constexpr int kStages = 4;      // units of a warp's ring
constexpr int kLeast = 4;       // units a CTA takes at least
// Units that a tile's start and end are worth in sharing out (64 sequences of 130
// to 8191 positions: 99 us with 0, 84 with 4, 81 with 8, 77 with 12, 78 with 20).
constexpr int kStart = 12;
constexpr int kSms = 152;       // the workspace holds the parts of as many SMs' CTAs
constexpr long long kMostUnits = 1ll << 38;  // of a call: below 2^31 a CTA of a full grid
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kMost = 256.f;  // a weight, or weight times step, that is let pass (1 where it was the largest)

template <int HD>
constexpr int kStageBytes = kUnit * HD + 2 * kUnit * 4;  // codes of k and v, scales of k and v
template <int HD>
constexpr int kSmem = kWarps * kStages * kStageBytes<HD>;
template <int NT>
constexpr int kResident = NT == 1 ? 3 : 2;  // CTAs of an SM (four of 128 registers spilled: 64 ragged sequences 80 us, three 69, two 75)

struct Kv4Shape {
  FastDiv by_heads, by_rep;
  long long most;  // units of sequences that do not overlap (kMostUnits at most)
};

// The workspace: of every CTA two parts (its first tile's and its last's), each
// R rows of HD sums, R maxima (log2 units) and R sums of weights; then a word
// pair for every row and query head: the first CTA that holds a part of it; how
// many more do (<< 6), which of that CTA's two it is (<< 5; the others' first)
// and the row's place in its tile.
struct Kv4Ws {
  float* part;
  int2* where;
};
template <int HD, int R>
constexpr int kPartFloats = R * (HD + 2);

__device__ __forceinline__ uint32_t transposed(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

// Row tiles of sequence b and the units of each (0 behind the last sequence).
// In sharing out a tile counts kStart more, in front: what its start and end
// take (short contexts else keep their CTAs longest).
struct Load {
  int tiles, units;
};
__device__ __forceinline__ Load seq_load(const PackedArgs& a, int cap, int rep, int rows, int b) {
  if (b >= a.B) return Load{0, 0};
  const int n = max(0, min(__ldg(a.kv_len + b), cap));
  return Load{(int)(((long long)seq_span(a, b, false).n * rep + rows - 1) / rows), (n + kUnit - 1) / kUnit};
}

__device__ __forceinline__ void cp_wait_stages() { asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory"); }
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

template <int HD, bool F16, int NT>
__global__ void __launch_bounds__(kThreads, kResident<NT>)
    k_kv4_attn(const __grid_constant__ PackedArgs a, const __grid_constant__ Kv4Args c, const __grid_constant__ Kv4Shape sh, Kv4Ws ws) {
  constexpr int NST = kStages, SB = kStageBytes<HD>, R = 8 * NT, KW = HD / 32;  // KW: words of k's codes a lane takes
  constexpr uint32_t kLow = 0x000f000fu, kHigh = 0x00f000f0u;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ float s_m[kWarps][R], s_l[kWarps][R];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  check_start(a);
  const int rep = sh.by_rep.d, cap = c.width << c.page_log, in_page = (1 << c.page_log) - 1;
  if (blockIdx.x == 0 && a.err)
    for (int b = tid; b < a.B; b += kThreads) {
      const int len = __ldg(a.kv_len + b);
      seq_span(a, b, true);
      if (len < 0 || len > cap) atomicOr(a.err, RL_DEVERR_CAPACITY);
    }
  // the batch's units, and this CTA's share of them
  long long all = 0;
  for (int b0 = 0; b0 < a.B; b0 += 32) {
    const Load x = seq_load(a, cap, rep, R, b0 + lane);
    all += x.units ? (long long)x.tiles * (x.units + kStart) : 0;
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) all += __shfl_xor_sync(0xffffffffu, all, d);
  all *= a.Hkv;
  if (all > sh.most) {  // (sequences overlap: not computed)
    if (tid == 0 && a.err) atomicOr(a.err, RL_DEVERR_CAPACITY);
    return;
  }
  const long long ctas = max(1ll, min((long long)gridDim.x, all / (kStart + kLeast)));
  const long long at = all * blockIdx.x / ctas, stop_at = blockIdx.x < ctas ? all * (blockIdx.x + 1) / ctas : 0;
  if (at >= stop_at) return;
  __shared__ long long s_all, s_ctas, s_stop;  // (needed at a tile's end only)
  if (tid == 0) {
    s_all = all;
    s_ctas = ctas;
    s_stop = stop_at;
  }
  int left = (int)(stop_at - at);  // units of the share to come
  // the sequence, tile and head, and unit it starts with
  int b = 0, item = 0, u0 = 0;
  Load ld{0, 0};
  {
    long long before = 0;
    for (int b0 = 0; b0 < a.B; b0 += 32) {
      const Load x = seq_load(a, cap, rep, R, b0 + lane);
      const long long mine = x.units ? (long long)x.tiles * (x.units + kStart) * a.Hkv : 0;
      long long sum = mine;  // of this lane's sequence and those in front
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, sum, d);
        if (lane >= d) sum += y;
      }
      const unsigned it = __ballot_sync(0xffffffffu, before + sum > at);
      if (it) {
        const int who = __ffs(it) - 1;
        b = b0 + who;
        ld.tiles = __shfl_sync(0xffffffffu, x.tiles, who);
        ld.units = __shfl_sync(0xffffffffu, x.units, who);
        const long long rest = at - before - __shfl_sync(0xffffffffu, sum - mine, who);
        item = (int)(rest / (ld.units + kStart));
        u0 = (int)(rest - (long long)item * (ld.units + kStart)) - kStart;
        break;
      }
      before += __shfl_sync(0xffffffffu, sum, 31);
    }
  }
  unsigned char* const ring = smem + warp * NST * SB;
  for (bool head_part = true;; head_part = false) {
    const int u1 = min(ld.units, u0 + left);
    if (u1 <= 0) break;  // (the share ends before the tile's first unit)
    left += min(u0, 0);
    u0 = max(u0, 0);
    const int tile = sh.by_heads.quot(item), hk = item - tile * sh.by_heads.d, row0 = tile * R;
    const Span sp = seq_span(a, b, false);
    const int old = max(0, min(__ldg(a.kv_len + b), cap)) - sp.all;  // position of the sequence's first row here
    const int nrow = min(R, sp.n * rep - row0);
    // keys that every row sees, and that any row sees
    const int every = old + sh.by_rep.quot(row0) + 1, any = max(0, old + sh.by_rep.quot(row0 + nrow - 1) + 1);
    const int units = min(u1, (any + kUnit - 1) / kUnit);

    // this lane's 16-byte pieces of a unit: of k's and v's codes every 512 bytes,
    // and (lanes 0-15) one of the scales
    const int head0 = hk << c.page_log;  // the head's first row in a page
    const bool v_scales = lane & 8;
    const unsigned char* const sc0 = reinterpret_cast<const unsigned char*>((v_scales ? c.vm : c.km) + head0) + (lane & 3) * 16;
    const unsigned sc_step = 4u * (unsigned)(v_scales ? c.vm_step : c.km_step), kc_step = (unsigned)c.kc_step, vc_step = (unsigned)c.vc_step;
    const uint32_t dst0 = smem_u32(ring) + lane * 16;
    // Pages: lane i has that of the (i % 2)-th 16 keys of this warp's unit number
    // k0 + i / 2 (of keys that nobody sees: some page of the sequence).
    int pages = 0;
    auto look_up = [&](int k0) {
      const int j = max(0, min((u0 + warp + (k0 + (lane >> 1)) * kWarps) * kUnit + (lane & 1) * 16, any - 1));
      pages = __ldg(c.table + (long long)b * c.table_step + (j >> c.page_log));
      if ((unsigned)pages >= (unsigned)c.n_pages) {  // out of the cache: reported, page 0 is read
        if (a.err) atomicOr(a.err, RL_DEVERR_CAPACITY);
        pages = 0;
      }
    };
    auto copy = [&](uint32_t dst, const unsigned char* src) {
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    };
    auto issue = [&](int k, int st) {  // this warp's k-th unit
      if ((k & 15) == 0) look_up(k);
      const int u = u0 + warp + k * kWarps;
      const unsigned px = __shfl_sync(0xffffffffu, pages, 2 * k & 31), py = __shfl_sync(0xffffffffu, pages, (2 * k & 31) | 1);
      if (u < units) {
        constexpr int NI = HD / 64;  // pieces of 16 keys
        const int r0 = (u * kUnit) & in_page, r1 = (u * kUnit + 16) & in_page;
        const int o0 = (head0 + r0) * (HD / 2) + lane * 16, o1 = (head0 + r1) * (HD / 2) + lane * 16;
        const uint32_t d = dst0 + st * SB;
        const unsigned char *k0 = c.kc + (size_t)px * kc_step + o0, *k1 = c.kc + (size_t)py * kc_step + o1;
        const unsigned char *v0 = c.vc + (size_t)px * vc_step + o0, *v1 = c.vc + (size_t)py * vc_step + o1;
  #pragma unroll
        for (int i = 0; i < NI; ++i) {
          copy(d + i * 512, k0 + i * 512);
          copy(d + (NI + i) * 512, k1 + i * 512);
          copy(d + kUnit * HD / 2 + i * 512, v0 + i * 512);
          copy(d + kUnit * HD / 2 + (NI + i) * 512, v1 + i * 512);
        }
        if (lane < 16) copy(d + kUnit * HD, sc0 + (size_t)(lane & 4 ? py : px) * sc_step + (lane & 4 ? r1 : r0) * 4);
      }
      cp_commit();
    };
  #pragma unroll
    for (int i = 0; i < NST - 1; ++i) issue(i, i);

    // B operands of q: this lane has row g of each tile, dims 32 t (16 t) and on
    uint32_t qb[NT][2 * KW][2];
    float mul[NT][2], qsum[NT][2];  // of the rows 2 t and 2 t + 1: scores are acc mul s + qsum m
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
      }
    }

    auto end_of = [&](int nt, int r) { return old + sh.by_rep.quot(row0 + nt * 8 + 2 * t + r) + 1; };  // keys a row sees
    float o[NT][HD / 16][4], o8[NT][4];  // sums over codes: dims (rows) g and g + 8 of a tile, query rows 2 t, 2 t + 1
    float m[NT][2], l[NT][2], z[NT][2];
    float base[NT][2], rel[NT][2];  // what scores are taken from, pivot(m); 2^(m - M): takes a weight times a step below 2^8
  #pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
  #pragma unroll
      for (int i = 0; i < HD / 16; ++i) o[nt][i][0] = o[nt][i][1] = o[nt][i][2] = o[nt][i][3] = 0.f;
      o8[nt][0] = o8[nt][1] = o8[nt][2] = o8[nt][3] = 0.f;
  #pragma unroll
      for (int r = 0; r < 2; ++r) {
        m[nt][r] = -INFINITY;
        l[nt][r] = z[nt][r] = base[nt][r] = rel[nt][r] = 0.f;
      }
    }
    // Key of a tile's row g: neighbours swapped in every second pair, so that the
    // loads of k (rows g, lanes t) and of v (rows 2 t, 2 t + 1, lanes g) both
    // spread over the banks.
    const int kg = g ^ ((g >> 1) & 1), ka = (2 * t) ^ (t & 1), kb = ka ^ 1;
    bool force = true;  // a row has no maximum yet
    int st = 0, st_in = NST - 1;
    for (int k = NST - 1, u = u0 + warp; u < units; u += kWarps, ++k) {
      cp_wait_stages();
      __syncwarp();  // everybody's copies have landed, and everybody is done with the stage before
      issue(k, st_in);
      st_in = st;
      const unsigned char* sk = ring + st * SB;
      const unsigned char* sv = sk + kUnit * HD / 2;
      const uint32_t* sm = reinterpret_cast<const uint32_t*>(sk + kUnit * HD);
      const int j0 = u * kUnit;
      const bool cut = j0 + kUnit > every;
      // scores from `base` on, weights, weights times v's steps; of keys g, g + 8:
      // v's step and m + 8 s
      float s[2][NT][4], w[2][NT][4], ws_[2][NT][4], vs[2][2], vm8[2][2];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        uint32_t x[2][KW];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const unsigned char* src = sk + (q * 16 + h * 8 + kg) * (HD / 2) + t * (HD / 8);
          if constexpr (HD == 128) {
            const uint4 v = *reinterpret_cast<const uint4*>(src);
            x[h][0] = v.x;
            x[h][1] = v.y;
            x[h][2] = v.z;
            x[h][3] = v.w;
          } else {
            const uint2 v = *reinterpret_cast<const uint2*>(src);
            x[h][0] = v.x;
            x[h][1] = v.y;
          }
        }
        float acc[NT][4] = {}, acc2[NT][4] = {};  // (two chains of products)
#pragma unroll
        for (int i = 0; i < KW; ++i) {
          const uint32_t x0 = x[0][i] >> 8, x1 = x[1][i] >> 8;
          const uint32_t lo[4] = {x[0][i] & kLow, x[1][i] & kLow, x[0][i] & kHigh, x[1][i] & kHigh};
          const uint32_t hi[4] = {x0 & kLow, x1 & kLow, x0 & kHigh, x1 & kHigh};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma_f16(acc[nt], lo[0], lo[1], lo[2], lo[3], qb[nt][2 * i][0], qb[nt][2 * i][1]);
            mma_f16(acc2[nt], hi[0], hi[1], hi[2], hi[3], qb[nt][2 * i + 1][0], qb[nt][2 * i + 1][1]);
          }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[nt][e] += acc2[nt][e];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int key = q * 16 + h * 8 + kg;
          const float2 km = unpack2<F16>(sm[key]), vm = unpack2<F16>(sm[kUnit + key]);
          vs[q][h] = vm.x;
          vm8[q][h] = fmaf(8.f, vm.x, vm.y);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int r = 0; r < 2; ++r)
              s[q][nt][2 * h + r] = fmaf(acc[nt][2 * h + r] * mul[nt][r], km.x, fmaf(km.y, qsum[nt][r], -base[nt][r]));
        }
      }
      if (cut) {
        asm volatile("");  // (a branch: as selects it cost every unit 16 of them)
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (j0 + q * 16 + (e >> 1) * 8 + kg >= end_of(nt, e & 1)) s[q][nt][e] = -INFINITY;
      }
      float most = 0.f;
      auto weigh = [&] {
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              w[q][nt][e] = ex2(s[q][nt][e]);
              ws_[q][nt][e] = w[q][nt][e] * rel[nt][e & 1] * vs[q][e >> 1];  // (in this order nothing overflows that the result holds)
              most = fmaxf(most, fmaxf(w[q][nt][e], fabsf(ws_[q][nt][e])));  // (a step may be below 0)
            }
      };
      weigh();
      if (__any_sync(0xffffffffu, most > kMost) || force) {
        // (seldom) new maxima of the rows, of weights and of weights times steps
        force = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float fo[2];
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            float x = -INFINITY, y = -INFINITY;
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                x = fmaxf(x, s[q][nt][2 * h + r]);
                y = fmaxf(y, s[q][nt][2 * h + r] + log2f(fabsf(vs[q][h])));
              }
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) {
              x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
              y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, d));
            }
            const float mn = fmaxf(m[nt][r], x + base[nt][r]), to = mn == -INFINITY ? 0.f : mn, f = ex2(m[nt][r] - to);
            const float M = rel[nt][r] == 0.f ? -INFINITY : base[nt][r] - log2f(rel[nt][r]);
            float Mn = fmaxf(M, y + base[nt][r]);
            // at least 2^-100 of the largest weight: as good as nothing, and a start while all steps so far are 0
            if (mn != -INFINITY) Mn = fmaxf(Mn, to - 100.f);
            fo[r] = M == -INFINITY ? 0.f : ex2(M - Mn);
            l[nt][r] *= f;
            z[nt][r] *= f;
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
              for (int h = 0; h < 2; ++h) s[q][nt][2 * h + r] += base[nt][r] - to;
            m[nt][r] = mn;
            base[nt][r] = to;
            rel[nt][r] = Mn == -INFINITY ? 0.f : ex2(to - Mn);
            force = force || mn == -INFINITY;
          }
#pragma unroll
          for (int i = 0; i < HD / 16; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[nt][i][e] *= fo[e & 1];
#pragma unroll
          for (int e = 0; e < 4; ++e) o8[nt][e] *= fo[e & 1];
        }
        force = __any_sync(0xffffffffu, force);
        weigh();
      }
      if (cut) {  // a key that a row does not see may hold anything
        asm volatile("");
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const bool see = j0 + q * 16 + (e >> 1) * 8 + kg < end_of(nt, e & 1);
              if (see) z[nt][e & 1] = fmaf(w[q][nt][e], vm8[q][e >> 1], z[nt][e & 1]);
              if (!see) ws_[q][nt][e] = 0.f;
            }
      } else {
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) z[nt][e & 1] = fmaf(w[q][nt][e], vm8[q][e >> 1], z[nt][e & 1]);
      }
      uint32_t p[2][NT][2];  // B operands: weights times steps
#pragma unroll
      for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int e = 0; e < 4; ++e) l[nt][e & 1] += w[q][nt][e];
          p[q][nt][0] = transposed(pack2<true>(ws_[q][nt][0], ws_[q][nt][1]));
          p[q][nt][1] = transposed(pack2<true>(ws_[q][nt][2], ws_[q][nt][3]));
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
      if (++st == NST) st = 0;
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
        const float f = rel[nt][r] == 0.f ? 0.f : 1.f / rel[nt][r];  // 2^(M - m): steps of 2^124 leave it finite
        const int row = nt * 8 + 2 * t + r;
  #pragma unroll
        for (int i = 0; i < HD / 16; ++i) {
          const float even = (o[nt][i][r] - o8[nt][r]) * 16777216.f, odd = (o[nt][i][2 + r] - 16.f * o8[nt][r]) * 1048576.f;
          *reinterpret_cast<float2*>(so + row * HD + g * (HD / 8) + 2 * i) = make_float2(fmaf(even, f, z[nt][r]), fmaf(odd, f, z[nt][r]));
        }
        if (g == 0) {
          s_m[warp][row] = m[nt][r];
          s_l[warp][row] = l[nt][r];
        }
      }
    __syncthreads();
    // The tile's rows, one a warp, lane with dims 2 lane + 64 i: finished here if
    // all of its units were, else a part.
    const bool whole = u0 == 0 && u1 == ld.units;
    float* const part = ws.part + ((long long)blockIdx.x * 2 + !head_part) * kPartFloats<HD, R>;
    for (int r = warp; r < nrow; r += kWarps) {
      float top = -INFINITY, sum = 0.f;
      for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_m[w][r]);
      float2 acc[HD / 64];
  #pragma unroll
      for (int i = 0; i < HD / 64; ++i) acc[i] = make_float2(0.f, 0.f);
  #pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = s_m[w][r] == -INFINITY ? 0.f : ex2(s_m[w][r] - top);
        // a state without keys has sum 0 (NaN of NaN scores: kept)
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
      const int i = row0 + r, tq = sh.by_rep.quot(i);
      const long long n = sp.first + tq, h = hk * rep + i - tq * rep;
      if (whole) {
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        uint16_t* o = static_cast<uint16_t*>(a.out) + n * a.os[0] + h * a.os[1] + 2 * lane;
  #pragma unroll
        for (int e = 0; e < HD / 64; ++e) *reinterpret_cast<uint32_t*>(o + 64 * e) = pack2<F16>(acc[e].x * inv, acc[e].y * inv);
        if (lane == 0 && a.lse) a.lse[n * a.Hq + h] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
      } else {
  #pragma unroll
        for (int e = 0; e < HD / 64; ++e) *reinterpret_cast<float2*>(part + r * HD + 2 * lane + 64 * e) = acc[e];
        if (lane == 0) {
          part[R * HD + r] = top;
          part[R * HD + R + r] = sum;
        }
      }
      if (u0 == 0 && lane == 0) {  // (the CTA of unit x is that of the largest i with i all / ctas <= x)
        const int end_cta = whole ? blockIdx.x : (int)(((s_stop - left + ld.units) * s_ctas - 1) / s_all);
        ws.where[n * a.Hq + h] = make_int2(blockIdx.x, (end_cta - (int)blockIdx.x) << 6 | !head_part << 5 | r);
      }
    }
    left -= u1 - u0;
    if (left <= 0) break;
    // the next tile: of this sequence, or of the next with any
    u0 = -kStart;
    if (++item == ld.tiles * a.Hkv) {
      item = 0;
      do ld = seq_load(a, cap, rep, R, ++b);
      while (b < a.B && (ld.tiles == 0 || ld.units == 0));  // (the end: only if lengths change meanwhile)
    }
    __syncthreads();  // (the rings are free)
  }
}

// A CTA a row and query head: its parts, a warp every fourth; rows without a key.
template <int HD, bool F16, int R>
__global__ void __launch_bounds__(128) k_kv4_join(const __grid_constant__ PackedArgs a, Kv4Ws ws, FastDiv by_heads, int ctas) {
  __shared__ float s_m[4], s_l[4], s_o[4][HD];
  const int n = by_heads.quot(blockIdx.x), h = blockIdx.x - n * a.Hq;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = seq_of_row(a, n, lane);
  pdl_wait();  // (everybody: what follows on the stream may take the first kernel as complete, too)
  if (b < 0) return;
  const Span sp = seq_span(a, b, false);
  if (n - sp.first >= sp.n) return;
  uint16_t* out = static_cast<uint16_t*>(a.out) + n * a.os[0] + h * a.os[1] + 2 * lane;
  if (__ldg(a.kv_len + b) <= 0) {
    if (warp == 0) {
#pragma unroll
      for (int e = 0; e < HD / 64; ++e) *reinterpret_cast<uint32_t*>(out + 64 * e) = 0u;
      if (lane == 0 && a.lse) a.lse[(long long)n * a.Hq + h] = -INFINITY;
    }
    return;
  }
  const int2 where = ws.where[(long long)n * a.Hq + h];
  const int parts = min((where.y >> 6) + 1, ctas), r = where.y & (R - 1);  // (bounds: nothing was written for starts that overlap)
  if (parts <= 1) return;
  auto at = [&](int i) { return ws.part + ((long long)min((unsigned)(where.x + i), (unsigned)ctas - 1) * 2 + (i == 0 ? where.y >> 5 & 1 : 0)) * kPartFloats<HD, R>; };
  float top = -INFINITY, sum = 0.f;
  float2 acc[HD / 64];
#pragma unroll
  for (int e = 0; e < HD / 64; ++e) acc[e] = make_float2(0.f, 0.f);
  for (int i0 = warp; i0 < parts; i0 += 16) {  // four parts' loads in flight together
    float m[4], l[4];
    float2 v[4][HD / 64];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int i = min(i0 + 4 * q, parts - 1);
      const float* p = at(i);
      m[q] = i0 + 4 * q < parts ? p[R * HD + r] : -INFINITY;
      l[q] = i0 + 4 * q < parts ? p[R * HD + R + r] : 0.f;
#pragma unroll
      for (int e = 0; e < HD / 64; ++e) v[q][e] = *reinterpret_cast<const float2*>(p + r * HD + 2 * lane + 64 * e);
    }
    const float mx = fmaxf(fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])), top);
    const float f0 = top == -INFINITY ? 0.f : ex2(top - mx);
    sum *= top == -INFINITY ? 1.f : f0;
#pragma unroll
    for (int e = 0; e < HD / 64; ++e) {
      acc[e].x *= f0;
      acc[e].y *= f0;
    }
    top = mx;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float f = m[q] == -INFINITY ? 0.f : ex2(m[q] - top);
      sum += m[q] == -INFINITY ? l[q] : f * l[q];
      if (f != 0.f) {
#pragma unroll
        for (int e = 0; e < HD / 64; ++e) {
          acc[e].x += f * v[q][e].x;
          acc[e].y += f * v[q][e].y;
        }
      }
    }
  }
#pragma unroll
  for (int e = 0; e < HD / 64; ++e) *reinterpret_cast<float2*>(&s_o[warp][2 * lane + 64 * e]) = acc[e];
  if (lane == 0) {
    s_m[warp] = top;
    s_l[warp] = sum;
  }
  __syncthreads();
  if (warp != 0) return;
  top = fmaxf(fmaxf(s_m[0], s_m[1]), fmaxf(s_m[2], s_m[3]));
  sum = 0.f;
#pragma unroll
  for (int e = 0; e < HD / 64; ++e) acc[e] = make_float2(0.f, 0.f);
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const float f = s_m[w] == -INFINITY ? 0.f : ex2(s_m[w] - top);
    sum += s_m[w] == -INFINITY ? s_l[w] : f * s_l[w];
    if (f != 0.f) {
#pragma unroll
      for (int e = 0; e < HD / 64; ++e) {
        const float2 v = *reinterpret_cast<const float2*>(&s_o[w][2 * lane + 64 * e]);
        acc[e].x += f * v.x;
        acc[e].y += f * v.y;
      }
    }
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
  for (int e = 0; e < HD / 64; ++e) *reinterpret_cast<uint32_t*>(out + 64 * e) = pack2<F16>(acc[e].x * inv, acc[e].y * inv);
  if (lane == 0 && a.lse) a.lse[(long long)n * a.Hq + h] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
}

// Units there can be, with row tiles of `rows` rows.
long long most_units(const PackedArgs& p, const Kv4Args& c, int rows) {
  const long long units = (((long long)c.width << c.page_log) + kUnit - 1) / kUnit;
  const long long n = p.start ? min((long long)p.max_rows * p.B, (long long)p.N) : p.B;
  return ((n * (p.Hq / p.Hkv) + rows - 1) / rows + p.B) * p.Hkv * (units + kStart);
}

template <int HD, bool F16, int NT>
cudaError_t launch(const PackedArgs& p, const Kv4Args& c, void* d_ws, cudaStream_t s) {
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
      if (e != cudaSuccess) return e;
      done[dev] = true;
    }
  }
  Kv4Ws ws;
  ws.where = static_cast<int2*>(d_ws);
  ws.part = static_cast<float*>(d_ws) + 2ll * p.N * p.Hq;
  // no more CTAs than units there can be
  const long long most = most_units(p, c, 8 * NT);
  const int grid = (int)min((long long)kResident<NT> * min(sms, kSms), (most + kLeast - 1) / kLeast);
  kern<<<grid, kThreads, kSmem<HD>, s>>>(p, c, Kv4Shape{FastDiv(p.Hkv), FastDiv(p.Hq / p.Hkv), most}, ws);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.N * p.Hq);
  cfg.blockDim = dim3(128);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_kv4_join<HD, F16, 8 * NT>, p, ws, FastDiv(p.Hq), grid);
}

// One tile of 8 rows, or two to an operand of codes: with more than 8 rows of a
// KV head a sequence (that share its keys) the second saves reading them again.
int row_tiles(const PackedArgs& p) { return (long long)(p.start ? p.max_rows : 1) * (p.Hq / p.Hkv) <= 8 ? 1 : 2; }

template <int HD, bool F16>
cudaError_t launch_rows(const PackedArgs& p, const Kv4Args& c, void* ws, cudaStream_t s) {
  return row_tiles(p) == 1 ? launch<HD, F16, 1>(p, c, ws, s) : launch<HD, F16, 2>(p, c, ws, s);
}

}  // namespace

bool kv4_attention_fits(const PackedArgs& p, const Kv4Args& c) { return most_units(p, c, 8 * row_tiles(p)) <= kMostUnits; }

size_t kv4_attention_ws_bytes(const PackedArgs& p) {
  static_assert(kResident<1> * 8 <= kResident<2> * 16, "the larger of the two forms");
  return 8ull * p.N * p.Hq + 2ull * kSms * kResident<2> * 16 * (p.hd + 2) * sizeof(float);
}

cudaError_t launch_kv4_attention(const PackedArgs& p, const Kv4Args& c, void* ws, cudaStream_t s) {
  if (p.hd == 64) return p.f16 ? launch_rows<64, true>(p, c, ws, s) : launch_rows<64, false>(p, c, ws, s);
  return p.f16 ? launch_rows<128, true>(p, c, ws, s) : launch_rows<128, false>(p, c, ws, s);
}

}  // namespace river

using namespace river;

extern "C" rl_status rl_kv4_attention_workspace(const rl_packed_desc* p, uint64_t* bytes) {
  const char* who = "rl_kv4_attention_workspace";
  PackedArgs a;
  const rl_status st = check_packed(who, p, kUsesQ, kUsesOut, &a);
  if (st != RL_OK) return st;
  if (!bytes) return op_error(who, RL_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = kv4_attention_ws_bytes(a);
  return RL_OK;
}

extern "C" rl_status rl_kv4_attention(const rl_kv4* c, const rl_packed_desc* p, const int32_t* d_start, const int32_t* d_kv_len,
                                      const void* d_q, void* d_out, float* d_lse, void* d_ws, uint64_t ws_bytes, int32_t* d_err,
                                      rl_stream_t stream) {
  const char* who = "rl_kv4_attention";
  PackedArgs a;
  Kv4Args k;
  rl_status st = check_packed(who, p, kUsesQ, kUsesOut, &a);
  if (st == RL_OK) st = check_kv4(who, c, a, &k);
  if (st != RL_OK) return st;
  if (!d_kv_len || !d_q || !d_out || d_out == d_q) return op_error(who, RL_ERR_INVALID_ARG, "NULL argument, or out in q's place");
  if (!d_start && p->rows != p->batch) return op_error(who, RL_ERR_INVALID_ARG, "rows must be batch without d_start");
  if (!op_aligned16(d_q) || !op_aligned16(d_out) || !op_aligned16(d_ws))
    return op_error(who, RL_ERR_UNSUPPORTED, "q, out and the workspace must start on 16-byte boundaries");
  if (!d_ws || ws_bytes < kv4_attention_ws_bytes(a)) return op_error(who, RL_ERR_INVALID_ARG, "workspace NULL or too small");
  a.q = d_q;
  a.out = d_out;
  a.lse = d_lse;
  a.start = d_start;
  a.kv_len = d_kv_len;
  a.err = d_err;
  if (!kv4_attention_fits(a, k)) return op_error(who, RL_ERR_UNSUPPORTED, "rows, table_width and heads make more than 2^38 units of 32 keys");
  const cudaError_t e = launch_kv4_attention(a, k, d_ws, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return set_error(RL_ERR_CUDA, cudaGetErrorString(e));
  return RL_OK;
}
