// Many query rows against one key range on the 5th-generation tensor cores:
// prompts under a sliding window, and the rows of all sequences against a
// shared prefix.
//
// A CTA takes 256 query rows (query position x the heads that share a KV
// head; for a prefix, sequence x those heads) as two M = 128 tiles and walks
// the keys any of them sees in tiles of 128:
//   S = Q K^T          tcgen05.mma, Q and K in shared memory, S in TMEM
//   w = exp2(S - m)    one thread a row; w rounded to the cache's type, in TMEM over S
//   O += w V           tcgen05.mma, w from TMEM, V as it lies ([key][dim]: the
//                      N-major operand), O in TMEM
// The two tiles share every K and V tile in shared memory (one alone would
// need 64 bytes a clock from L2 at the tensor cores' rate) and alternate: while
// one's rows are in the softmax the other's products run.
//   warps 0-3, 4-7  softmax of tile 0 and 1      warp 8  TMA (K, V in turn)
//   warp 9          MMA issue                    warps 10, 11  no work of their
//   own: setmaxnreg counts whole warpgroups
// A softmax thread holds its row's 128 scores in registers: of the 168 a
// thread the launch has, the control warps give most to them (216 + 216 + 72
// = 3 x 168; with 168 they spilled, and a tile pair took 5900 clocks, not 3300).
//
// What bounds it (8192 queries, window 2048, 32 heads, 8 KV heads, head_dim
// 128: 230 us, 0.56 of the measured bf16 rate; tensor pipe 45 % busy while a
// CTA runs): a row tile's chain.  Softmax 1600 clocks (maxima 470, the vote on
// rescaling 200, exponentials 820 of which the ex2 unit takes 512; a tile that
// a mask cuts 700 more), then the 16 products of its values and next scores
// (1345 from the first's issue to the last's arrival: 65 each behind 300), then
// two hand-offs; the two tiles of a CTA interleave to 3500 clocks a pair of
// tiles, in which the tensor cores could do 54 products and do 32.  The rest
// is CTAs' starts (4800 clocks to the first scores, half of it the copies' way,
// before Q came from L2) and ends (5800 from the last weights on, and 1500 until
// the next one runs) of 75000.  At head_dim 64 a product still takes 63 clocks (N = 64), so the rate
// is half: 5 ragged prompts, window 500: 38 us.
// The running maximum follows lazily: O and the sum are rescaled only when a
// row's maximum grew by more than 2^8 since the last time (weights then stay
// below 2^8, far inside both types; the sum is fp32), so most tiles touch O
// with the tensor core alone.
//
// Keys are dealt out over a cluster of S CTAs when the row tiles alone do not
// fill the GPU; its CTAs join their (maximum, sum, O) through distributed
// shared memory in a fixed order.
#include <atomic>
#include <mutex>

#include "attn_ops.cuh"

namespace river {

namespace {

using namespace dev;
using namespace attn;

constexpr int kThreads = 384;
constexpr int kRowsCta = 256;
constexpr int kKeys = 128;       // keys of a tile
constexpr int kMaxSplit = 8;     // CTAs of a cluster (of 16, no more than 7 clusters fit the SMs at once)
constexpr int kSpin = 1 << 20;   // polls of a wait before it gives up (one that fails takes 1.3 us)
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLazy = 8.f;     // log2 growth of a maximum that is let pass

std::atomic<long long> g_wait_polls{-1};  // rl_debug_limit_waits (below 0: kSpin)

template <int HD>
constexpr int kTileBytes = kKeys * HD * 2;  // a Q, K or V tile: HD / 64 blocks of 128 rows x 128 bytes
template <int HD>
constexpr int kStages = HD == 128 ? 4 : 8;
template <int HD>
constexpr int kSmem = (2 + kStages<HD>)*kTileBytes<HD> + 1024;

// Shared-memory matrix descriptors, 128-byte swizzle: the low word holds the
// address / 16 (and the leading byte offset), the high word is constant.
//   K-major (Q, K): rows of 128 bytes, 8-row swizzle atoms 1024 bytes apart.
//   N-major (V): 64 elements of N a row, the next 64 one block (128 rows) on,
//   8 rows of K 1024 bytes apart.
constexpr uint32_t kDescHi = (1024 >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_k_major(uint32_t addr) { return ((addr & 0x3FFFFu) >> 4) | (1u << 16); }
__device__ __forceinline__ uint32_t desc_n_major(uint32_t addr) {
  return ((addr & 0x3FFFFu) >> 4) | ((uint32_t)((kKeys * 128) >> 4) << 16);
}
// kind::f16, fp32 accumulate, M = 128.
__host__ __device__ constexpr uint32_t idesc(bool f16, int n, bool b_n_major) {
  return (1u << 4) | (f16 ? 0u : (1u << 7) | (1u << 10)) | (b_n_major ? 1u << 16 : 0u) | ((uint32_t)(n >> 3) << 17) |
         ((uint32_t)(128 >> 4) << 24);
}
// Every lane calls these with the same operands and the one with `el` != 0
// issues: a single lane's branch would move each operand to the uniform
// registers anew (32 MMAs a tile pair then cost more issue time than tensor time).
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t id, uint32_t acc, uint32_t el) {
  asm volatile(
      "{\n .reg .pred p, e;\n .reg .b64 x, y;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 e, %5, 0;\n"
      " mov.b64 x, {%1, %6};\n mov.b64 y, {%2, %6};\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(id), "r"(acc), "r"(el), "r"(kDescHi)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t id, uint32_t acc, uint32_t el) {
  asm volatile(
      "{\n .reg .pred p, e;\n .reg .b64 y;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 e, %5, 0;\n"
      " mov.b64 y, {%2, %6};\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(id), "r"(acc), "r"(el), "r"(kDescHi)
      : "memory");
}
__device__ __forceinline__ void commit(uint64_t* bar, uint32_t el) {
  asm volatile(
      "{\n .reg .pred e;\n setp.ne.b32 e, %1, 0;\n"
      " @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(smem_u32(bar)),
      "r"(el)
      : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

#define RL_R8(r, i) "=f"(r[i]), "=f"(r[i + 1]), "=f"(r[i + 2]), "=f"(r[i + 3]), "=f"(r[i + 4]), "=f"(r[i + 5]), "=f"(r[i + 6]), "=f"(r[i + 7])
#define RL_I8(r, i) "r"(r[i]), "r"(r[i + 1]), "r"(r[i + 2]), "r"(r[i + 3]), "r"(r[i + 4]), "r"(r[i + 5]), "r"(r[i + 6]), "r"(r[i + 7])
// 32 consecutive fp32 columns of this thread's lane (complete after ld_wait).
__device__ __forceinline__ void tmem_ld32(uint32_t at, float* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : RL_R8(r, 0), RL_R8(r, 8), RL_R8(r, 16), RL_R8(r, 24)
      : "r"(at));
}
// Waits for this thread's TMEM loads; the values pass through, so that no use
// of them moves ahead of the wait.
template <int N>
__device__ __forceinline__ void ld_wait(float* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+f"(r[i]));
}
__device__ __forceinline__ void tmem_st32(uint32_t at, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(at),
      RL_I8(r, 0), RL_I8(r, 8), RL_I8(r, 16), RL_I8(r, 24)
      : "memory");
}
// A row tile of Q: 64-dim blocks of 128 rows (query row x heads of the group).
__device__ __forceinline__ void tma_load_q(void* dst, const CUtensorMap* map, int head, int row, int seq, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %3, %6}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(0), "r"(head), "r"(row), "r"(seq)
      : "memory");
}
__device__ __forceinline__ void prefetch_q(const CUtensorMap* map, int head, int row, int seq) {
  asm volatile("cp.async.bulk.prefetch.tensor.5d.L2.global.tile [%0, {%1, %2, %3, %1, %4}];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(0), "r"(head), "r"(row), "r"(seq)
               : "memory");
}
__device__ __forceinline__ void st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Bits 0 .. n - 1.
__device__ __forceinline__ uint32_t below(int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1; }
// Scores whose bit is 0 become -infinity (selects on bits: as 128 conditions
// they were branches, 6000 to 11000 clocks a masked tile).
__device__ __forceinline__ void keep_only(float* s, uint32_t bits) {
#pragma unroll
  for (int e = 0; e < 32; ++e) s[e] = (bits >> e) & 1u ? s[e] : -INFINITY;
}

// Two fp32 operations an instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  unsigned long long d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(d)
      : "l"(*reinterpret_cast<unsigned long long*>(&a)), "l"(*reinterpret_cast<unsigned long long*>(&b)),
        "l"(*reinterpret_cast<unsigned long long*>(&c)));
  return *reinterpret_cast<float2*>(&d);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  unsigned long long d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(d)
      : "l"(*reinterpret_cast<unsigned long long*>(&a)), "l"(*reinterpret_cast<unsigned long long*>(&b)));
  return *reinterpret_cast<float2*>(&d);
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// A launch's shape: divisors, and whether Q comes by TMA (its map's axes: 64
// dims, heads, query rows, 64-dim blocks, sequences; a box is a row tile).
struct RowsShape {
  int split, tiles, q_tma, apart;
  int ahead;  // clusters that run at once: the one this many on follows on these SMs
  int polls;  // of a wait before it gives up
  FastDiv by_split, by_heads, by_group, by_rep;  // CTAs of a cluster, KV heads, KV heads x sequences, heads a KV head
};

struct Bars {
  uint64_t s_full[2], p_full[2], o_full[2], full[8], empty[8], drain;
};

template <int HD, bool F16, bool PREFIX>
__global__ void __launch_bounds__(kThreads, 1)
    k_attn_rows_tc(const __grid_constant__ KvMaps maps, const __grid_constant__ CUtensorMap q_map,
                   const __grid_constant__ AttnOpArgs a, const __grid_constant__ RowsShape sh) {
  constexpr int NST = kStages<HD>, TB = kTileBytes<HD>;
  extern __shared__ unsigned char smem_dyn[];
  unsigned char* smem =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~(uintptr_t)1023);
  unsigned char* sq = smem;            // [2] Q tiles
  unsigned char* ring = smem + 2 * TB; // K_0, V_0, K_1, V_1, ...
  __shared__ __align__(8) Bars bar;
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_fail;
  __shared__ int s_loaded;  // K and V tiles copied (set where the copying ends)
  __shared__ float s_m[kRowsCta], s_l[kRowsCta];  // a row's maximum (log2 units) and sum

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // the kernel that takes the prefix's parts may start beside the last CTAs
  // (it waits for all of them before it reads the workspace)
  if (PREFIX) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (tid == kThreads - 1) {  // (a thread without work of its own)
    prefetch_map(&maps.k);
    prefetch_map(&maps.v);
    if (sh.q_tma) prefetch_map(&q_map);
  }
  const int split = sh.split, tiles = sh.tiles, rep = sh.by_rep.d;
  int id = sh.by_split.quot(blockIdx.x);
  const int part = blockIdx.x - id * split;
  if (!PREFIX && tid == kThreads - 1 && part == 0 && sh.q_tma) {
    // Q of the CTA that follows here into L2 (its first scores wait for Q: the
    // 8192-token prompt 238 -> 236 us, the ragged ones 38.4 -> 37.6)
    const int nid = id + sh.ahead, nback = sh.by_group.quot(nid), nrow0 = (tiles - 1 - nback) * kRowsCta;
    if (nback < tiles) {
      const int rest = nid - nback * sh.by_group.d, nb = sh.by_heads.quot(rest);
      for (int g = 0; g < 2; ++g) {
        const int t = sh.by_rep.quot(nrow0 + g * 128);
        if (t < a.Tq) prefetch_q(&q_map, (rest - nb * sh.by_heads.d) * rep, t, nb);
      }
    }
  }
  // later tiles of a prompt see more keys: first come, first served from the end
  const int back = sh.by_group.quot(id);
  const int row0 = (tiles - 1 - back) * kRowsCta;
  id -= back * sh.by_group.d;
  const int b = sh.by_heads.quot(id), hk = id - b * sh.by_heads.d;  // (b is 0 for a prefix)
  int n, ql, nrow, p0 = 0, lo = 0, hi, sink_end = 0;
  if constexpr (PREFIX) {
    n = hi = a.P;
    ql = a.B;
    nrow = min(kRowsCta, a.B * rep - row0);
  } else {
    const bool report = part == 0 && tid == 0 && hk == 0 && row0 == 0;
    const Lens len = seq_lens(a, b, report);
    n = len.n;
    ql = len.ql;
    nrow = min(kRowsCta, ql * rep - row0);
    if (nrow <= 0) return;  // (its whole cluster: the rows are the same)
    // keys any row sees: [0, sink_end) and [lo, hi)
    p0 = max(n - ql + sh.by_rep.quot(row0), 0);
    const int p1 = n - ql + sh.by_rep.quot(row0 + nrow - 1);
    hi = max(p1 + 1, 0);
    if (hi > 0) lo = max(0, p0 - a.window + 1);
    sink_end = min(a.sinks, lo);
    if (sink_end == lo) lo = sink_end = 0;
  }
  const int su = (sink_end + kKeys - 1) / kKeys;
  const int all = su + (hi - lo + kKeys - 1) / kKeys;
  // (all < 2^24: at most 2^30 keys, in two ranges)
  const int j0 = sh.by_split.quot(all * part), nt = sh.by_split.quot(all * (part + 1)) - j0;
  auto key0 = [&](int j) { return j < su ? j * kKeys : lo + (j - su) * kKeys; };
  auto count = [&](int j) { return min(kKeys, (j < su ? sink_end : hi) - key0(j)); };
  const int ngrp = nrow > 128 ? 2 : 1;

  auto load = [&](int i) {  // K (i even) or V tile i / 2 into its stage
    const int st = i % NST, j = key0(j0 + (i >> 1));
    mbar_expect_tx(&bar.full[st], i == 0 && sh.q_tma ? (1 + ngrp) * TB : TB);
    if (i & 1)
      tma_load_5d(ring + st * TB, &maps.v, j, hk * maps.vh, b * maps.vb, &bar.full[st]);
    else
      tma_load_5d(ring + st * TB, &maps.k, j, hk * maps.kh, b * maps.kb, &bar.full[st]);
  };
  if (warp == 8) {
    if (lane == 0) {
      for (int i = 0; i < 2; ++i) {
        mbar_init(&bar.s_full[i], 1);
        mbar_init(&bar.p_full[i], 128);
        mbar_init(&bar.o_full[i], 1);
      }
      for (int i = 0; i < NST; ++i) {
        mbar_init(&bar.full[i], 1);
        mbar_init(&bar.empty[i], 1);
      }
      mbar_init(&bar.drain, 1);
      s_fail = 0;
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
      if (nt > 0) {
        load(0);  // (the others after Q's rows, which the first scores need too)
        if (sh.q_tma)
          for (int g = 0; g < ngrp; ++g) {
            const int t = sh.by_rep.quot(row0 + g * 128);
            tma_load_q(sq + g * TB, &q_map, hk * rep, t, b, &bar.full[0]);
          }
      }
    }
    __syncwarp();
  } else if (warp == 9) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)), "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  } else if (warp < 8 && warp / 4 < ngrp && nt > 0 && !sh.q_tma) {
    // Q rows to shared memory as the TMA would lay them; rows past the last are 0
    const int g = warp / 4, r = tid & 127;
    auto at = [&](int e) {  // 16-byte chunk e * 128 + r of the tile: its place in q
      const int it = e * 128 + r, i = row0 + min(g * 128 + it / (HD / 8), nrow - 1), t = sh.by_rep.quot(i);
      return (PREFIX ? (long long)t * a.qs[0] : (long long)b * a.qs[0] + (long long)t * a.qs[1]) +
             (long long)(hk * rep + i - t * rep) * a.qs[2] + it % (HD / 8) * 8;
    };
    auto put = [&](int e, uint4 v) {
      const int it = e * 128 + r, qr = it / (HD / 8), ch = it % (HD / 8);
      if (g * 128 + qr >= nrow) v = make_uint4(0, 0, 0, 0);
      *reinterpret_cast<uint4*>(sq + g * TB + (ch >> 3) * (128 * 128) + qr * 128 + (((ch & 7) ^ (qr & 7)) << 4)) = v;
    };
    if (a.q_f32) {
#pragma unroll 2
      for (int e = 0; e < HD / 8; ++e) {
        const float4* f = reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + at(e));
        const float4 x = __ldg(f), y = __ldg(f + 1);
        put(e, make_uint4(pack2<F16>(x.x, x.y), pack2<F16>(x.z, x.w), pack2<F16>(y.x, y.y), pack2<F16>(y.z, y.w)));
      }
    } else {
      uint4 v[HD / 8];  // all loads in flight before the first store
#pragma unroll
      for (int e = 0; e < HD / 8; ++e) v[e] = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + at(e)));
#pragma unroll
      for (int e = 0; e < HD / 8; ++e) put(e, v[e]);
    }
    fence_proxy_async_smem();
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = s_tmem;
  // false: gave up (this wait or another's); nobody computes any more
  auto wait = [&](uint64_t* w, uint32_t ph) {
    // (counted, not timed, and no more than this: a few instructions more here
    // cost the issuing warp's chain 8 % of a prompt's time)
    for (int i = 0; i < sh.polls; ++i) {
      if (mbar_try(w, ph)) return true;
      if ((i & 255) == 255 && s_fail) return false;
    }
    s_fail = 1;
    return false;
  };
  auto wait_warp = [&](uint64_t* w, uint32_t ph) { return __all_sync(0xffffffffu, wait(w, ph)) != 0; };
  // TMEM columns: S_0, S_1 (their weights over them), O_0, O_1
  auto t_s = [tmem](int g) { return tmem + g * 128; };
  auto t_o = [tmem](int g) { return tmem + 256 + g * 128; };

  if (warp >= 8) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
  if (warp == 8) {
    if (lane == 0) {
      int i = 1;
      for (; i < 2 * nt; ++i) {
        if (i >= NST && !wait(&bar.empty[i % NST], ((i / NST) - 1) & 1)) break;
        load(i);
      }
      s_loaded = nt > 0 ? i : 0;
    }
    __syncwarp();
  } else if (warp == 9) {
    if (nt > 0) {
      constexpr uint32_t idS = idesc(F16, kKeys, false), idO = idesc(F16, HD, true);
      const uint32_t el = lane == 0;
      const uint32_t q0 = desc_k_major(smem_u32(sq)), k0 = desc_k_major(smem_u32(ring)), v0 = desc_n_major(smem_u32(ring));
      auto scores = [&](int g, int j) {  // S_g = Q_g K_j^T
        const uint32_t q = q0 + g * (TB >> 4), k = k0 + ((2 * j) % NST) * (TB >> 4);
#pragma unroll
        for (int ks = 0; ks < HD / 16; ++ks) {
          const uint32_t off = (ks >> 2) * (kKeys * 128 >> 4) + (ks & 3) * 2;
          mma_ss(t_s(g), q + off, k + off, idS, ks != 0, el);
        }
        commit(&bar.s_full[g], el);
      };
      auto values = [&](int g, int j) {  // O_g += w_g V_j
        const uint32_t v = v0 + ((2 * j + 1) % NST) * (TB >> 4);
        mma_ts(t_o(g), t_s(g), v, idO, j != 0, el);
#pragma unroll
        for (int ks = 1; ks < kKeys / 16; ++ks) mma_ts(t_o(g), t_s(g) + ks * 8, v + ks * (2048 >> 4), idO, 1, el);
      };
      // (every lane polls; no vote: the waits are on the products' path)
      bool go = wait(&bar.full[0], 0);
      if (go) {
        scores(0, 0);
        if (ngrp == 2) scores(1, 0);
        commit(&bar.empty[0], el);
      }
      if (go) go = wait(&bar.full[1 % NST], 0) && (nt == 1 || wait(&bar.full[2 % NST], (2 / NST) & 1));
      for (int j = 0; j < nt && go; ++j) {
        const int iv = 2 * j + 1, ik = 2 * j + 2;
        const bool more = j + 1 < nt;
        if (!(go = wait(&bar.p_full[0], j & 1))) break;
        fence_after();
        values(0, j);
        if (more)
          scores(0, j + 1);
        else
          commit(&bar.o_full[0], el);
        if (ngrp == 2) {
          if (!(go = wait(&bar.p_full[1], j & 1))) break;
          fence_after();
          values(1, j);
        }
        commit(&bar.empty[iv % NST], el);
        if (more) {
          if (ngrp == 2) scores(1, j + 1);
          commit(&bar.empty[ik % NST], el);
          // the next tiles, while the products issued run
          go = wait(&bar.full[(iv + 2) % NST], ((iv + 2) / NST) & 1) &&
               (j + 2 >= nt || wait(&bar.full[(ik + 2) % NST], ((ik + 2) / NST) & 1));
        } else if (ngrp == 2) {
          commit(&bar.o_full[1], el);
        }
      }
      if (!go) {  // what was issued still completes before TMEM is given back
        commit(&bar.drain, el);
        mbar_wait(&bar.drain, 0, kSpin);
      }
    }
    __syncwarp();
  }

  const bool direct = PREFIX || split == 1;  // no other CTA's keys are joined here
  if (warp >= 8) {
    if (!direct) {  // (the softmax warps' two below)
      cluster_barrier();
      cluster_barrier();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    const int g = warp >> 2, r = tid & 127;  // softmax: tile and row
    float m = -INFINITY, l = 0.f;            // m in units of raw scores
    const float sc = a.scale * kLog2e;
    const uint32_t lane_at = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ts = t_s(g & 1), to = t_o(g & 1);
    const int i_row = row0 + g * 128 + r;    // (query, head in group)
    bool go = true;                          // (the same for a warp)
    if (g < ngrp && nt > 0) {
      const int p = PREFIX ? 0 : n - ql + sh.by_rep.quot(i_row);  // this row's position
      // positions of the tile's first and last row that count
      const int pa = PREFIX ? 0 : max(n - ql + sh.by_rep.quot(row0 + g * 128), 0);
      const int pz = PREFIX ? 0 : n - ql + sh.by_rep.quot(row0 + min(nrow, g * 128 + 128) - 1);
      // and of the warp's
      const int wr = row0 + g * 128 + (warp & 3) * 32;
      const int wa = PREFIX ? 0 : n - ql + sh.by_rep.quot(wr);
      const int wz = PREFIX ? 0 : n - ql + sh.by_rep.quot(wr + 31);
      for (int j = 0; j < nt; ++j) {
        const int k0 = key0(j0 + j), cnt = count(j0 + j);
        if (!(go = wait_warp(&bar.s_full[g], j & 1))) break;
        fence_after();
        float s[kKeys];
#pragma unroll
        for (int c = 0; c < kKeys; c += 32) tmem_ld32(ts + lane_at + c, s + c);
        ld_wait<kKeys>(s);
        if (PREFIX) {
          if (cnt < kKeys) {
#pragma unroll
            for (int c = 0; c < kKeys; c += 32)
              if (c + 32 > cnt) keep_only(s + c, below(cnt - c));
          }
        } else if (cnt < kKeys || k0 + kKeys - 1 > pa || (pz - k0 >= a.window && k0 + kKeys > a.sinks)) {
          // keys this row sees: below `end`, and from `beg` on or below `snk`
          const int end = min(cnt, p - k0 + 1), beg = p - a.window + 1 - k0, snk = a.sinks - k0;
#pragma unroll
          for (int c = 0; c < kKeys; c += 32) {
            // (a warp's rows have few positions: most groups of 32 keys are whole for all)
            const int k = k0 + c;
            if (c + 32 > cnt || k + 31 > wa || (wz - k >= a.window && k + 31 >= a.sinks))
              keep_only(s + c, below(end - c) & (~below(beg - c) | below(snk - c)));
          }
        }
        float x[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) x[c] = max3(s[c], s[c + 4], s[c + 8]);
#pragma unroll
        for (int c = 12; c + 8 <= kKeys; c += 8)
#pragma unroll
          for (int e = 0; e < 4; ++e) x[e] = max3(x[e], s[c + e], s[c + 4 + e]);
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = fmaxf(x[e], s[kKeys - 4 + e]);
        const float mx = fmaxf(max3(x[0], x[1], x[2]), x[3]);
        if (__any_sync(0xffffffffu, mx * sc > m * sc + kLazy || (m == -INFINITY && mx > m))) {
          const float mn = fmaxf(m, mx);
          const float f = m == -INFINITY ? 0.f : ex2((m - mn) * sc);
          l *= f;
          m = mn;
          if (j > 0) {
            // the products of the tiles before are complete (S_j was issued after them)
#pragma unroll
            for (int c = 0; c < HD; c += 32) {
              float o[32];
              uint32_t u[32];
              tmem_ld32(to + lane_at + c, o);
              ld_wait<32>(o);
#pragma unroll
              for (int e = 0; e < 32; ++e) u[e] = __float_as_uint(o[e] * f);
              tmem_st32(to + lane_at + c, u);
            }
          }
        }
        const float ms = m == -INFINITY ? 0.f : m * sc;
        float2 y[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        const float2 sc2 = make_float2(sc, sc), ms2 = make_float2(-ms, -ms);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t w[32];
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            float2 u = fma2(make_float2(s[h * 64 + 2 * c], s[h * 64 + 2 * c + 1]), sc2, ms2);
            u.x = ex2(u.x);
            u.y = ex2(u.y);
            y[c & 1] = add2(y[c & 1], u);
            w[c] = pack2<F16>(u.x, u.y);
          }
          tmem_st32(ts + lane_at + h * 32, w);
        }
        const float2 yy = add2(y[0], y[1]);
        l += yy.x + yy.y;
        // V rows behind the sequence or the sinks may hold anything: 0 * NaN must
        // not happen (a prefix has none; a NaN in keys of the window that only
        // other rows see is met at the end)
        const int from = PREFIX ? kKeys : j0 + j < su ? cnt : n - k0;
        if (from < kKeys) {
          const int iv = 2 * j + 1;
          if (!(go = wait_warp(&bar.full[iv % NST], (iv / NST) & 1))) break;
          unsigned char* sv = ring + (iv % NST) * TB;
          for (int it = tid & 127; it < (kKeys - from) * (HD / 8); it += 128) {
            const int kr = from + it / (HD / 8), ch = it % (HD / 8);
            *reinterpret_cast<uint4*>(sv + (ch >> 3) * (kKeys * 128) + kr * 128 + (ch & 7) * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
        }
        st_wait();
        fence_before();
        mbar_arrive(&bar.p_full[g]);
      }
    }
    const bool mine = g * 128 + r < nrow;
    long long row_at = -1;  // where the row's output goes
    float inv = 0.f;
    if (!PREFIX && direct && mine) {  // (while the last products run)
      const int t = sh.by_rep.quot(i_row), h = hk * rep + i_row - t * rep;
      row_at = b * a.os[0] + t * a.os[1] + h * a.os[2];
      inv = l == 0.f ? 0.f : 1.f / l;
      if (a.lse) a.lse[((long long)b * a.Tq + t) * a.Hq + h] = l == 0.f ? -INFINITY : (m * sc + log2f(l)) * 0.6931471805599453f;
    }
    if (g < ngrp && nt > 0) {
      // (the last tile's: the ring, which the other tile's products still read,
      // is written over below)
      if (!go || !(go = wait_warp(&bar.o_full[PREFIX || !direct ? ngrp - 1 : g], 0))) {
        l = inv = NAN;
        if (row_at >= 0 && a.lse) {  // (stored above, of the keys there were)
          const int t = sh.by_rep.quot(i_row);
          a.lse[((long long)b * a.Tq + t) * a.Hq + hk * rep + i_row - t * rep] = NAN;
        }
      }
      fence_after();
    }
    auto weight = [](float x, float top) { return x == -INFINITY ? 0.f : ex2(x - top); };
    {
      const bool have = g < ngrp && nt > 0;
      if constexpr (PREFIX) {
        // O, maximum and sum of the CTA's keys to the workspace, 32 rows a warp:
        // through shared memory over the drained ring (16-byte chunk c of row q
        // at c ^ (q mod chunks), and so in the workspace) by one bulk copy
        constexpr int CH = HD / 4;
        const int q0 = g * 128 + (warp & 3) * 32, rows = min(32, nrow - q0);
        if (have && rows > 0) {
          float4* dst = reinterpret_cast<float4*>(ring) + (q0 + lane) * CH;
#pragma unroll
          for (int c = 0; c < HD; c += 32) {
            float o[32];
            tmem_ld32(to + lane_at + c, o);
            ld_wait<32>(o);
#pragma unroll
            for (int e = 0; e < 32; e += 4) dst[((c + e) / 4) ^ (lane & (CH - 1))] = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
          }
          fence_proxy_async_smem();
          __syncwarp();
          const PrefixWs ws = prefix_ws(a.ws, row0 / kRowsCta, tiles, a.B * rep, hk, a.Hkv, part, split + sh.apart, HD);
          if (lane == 0) {
            bulk_s2g(ws.o + (long long)q0 * HD, ring + q0 * HD * 4, rows * HD * 4);
            asm volatile("cp.async.bulk.commit_group;\ncp.async.bulk.wait_group 0;" ::: "memory");
          }
          if (lane < rows) {
            ws.m[q0 + lane] = l == 0.f ? -INFINITY : m * sc;
            ws.l[q0 + lane] = l;
          }
        }
      } else if (direct) {
        const bool dead = !have || l == 0.f;  // (a row that sees no key: O may hold anything)
        float chk = 0.f;                      // NaN once a value is not finite
        // through shared memory (over Q, which no product reads any more), so that
        // whole rows are written, not 16 bytes of 32 rows at a time
        constexpr int CR = HD / 8;  // 16-byte chunks of a row; chunk c of row q at c ^ (q & 7)
        unsigned char* stage = sq + g * TB + (warp & 3) * (32 * HD * 2);
#pragma unroll
        for (int c = 0; c < HD; c += 32) {
          float o[32] = {};
          if (have) {
            tmem_ld32(to + lane_at + c, o);
            ld_wait<32>(o);
          }
#pragma unroll
          for (int e = 0; e < 32; e += 8) {
            uint32_t w[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const float u = o[e + 2 * q] * inv, v = o[e + 2 * q + 1] * inv;
              chk = fmaf(u, 0.f, fmaf(v, 0.f, chk));
              w[q] = dead ? 0u : pack2<F16>(u, v);
            }
            *reinterpret_cast<uint4*>(stage + lane * (HD * 2) + ((((c + e) / 8) ^ (lane & 7)) << 4)) =
                make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
        __syncwarp();
#pragma unroll 4
        for (int q = lane / CR; q < 32; q += 32 / CR) {
          const long long at = __shfl_sync(0xffffffffu, row_at, q);
          const int c = lane % CR;
          uint4 v = *reinterpret_cast<const uint4*>(stage + q * (HD * 2) + ((c ^ (q & 7)) << 4));
          // (after a wait that gave up Q's copy may land on the staged rows)
          if (!go) v = make_uint4(0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu);
          if (at >= 0) *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + at + c * 8) = v;
        }
        // rows of different masks shared V's tiles: one that is not finite may
        // owe that to a key it does not see (0 * infinity)
        unsigned bad = __ballot_sync(0xffffffffu, mine && !dead && chk != 0.f);
        if (__any_sync(0xffffffffu, s_fail)) bad = 0;  // (the same for every lane: exact_row shuffles)
        if (bad) __syncwarp();  // the rows' first values, stored by other lanes, come before the new ones
        while (bad) {
          const int i = row0 + g * 128 + (warp & 3) * 32 + __ffs(bad) - 1;
          bad &= bad - 1;
          const int ti = sh.by_rep.quot(i);
          exact_row<HD, F16>(a, b, ti, hk * rep + i - ti * rep, n, ql, lane);
        }
      } else {
        // to shared memory over the drained ring: rows of HD floats, 16-byte
        // chunk c of row q at c ^ (q mod chunks)
        constexpr int CH = HD / 4;
        s_m[g * 128 + r] = have && l != 0.f ? m * sc : -INFINITY;
        s_l[g * 128 + r] = l;
        if (have) {
          float4* dst = reinterpret_cast<float4*>(ring) + (g * 128 + r) * CH;
#pragma unroll
          for (int c = 0; c < HD; c += 32) {
            float o[32];
            tmem_ld32(to + lane_at + c, o);
            ld_wait<32>(o);
#pragma unroll
            for (int e = 0; e < 32; e += 4) dst[((c + e) / 4) ^ (r & (CH - 1))] = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
          }
        }
      }
    }
    if (!direct) {
      cluster_barrier();
      constexpr int CH = HD / 4;
      // one row a warp, dealt out over the cluster's warps 0 .. 7; lane has the
      // 16-byte chunk `lane` (HD 64: the lower 16 lanes)
      for (int q = part * 8 + warp; q < nrow; q += split * 8) {
        float cm = -INFINITY, cl = 0.f;
        if (lane < split) {
          cm = cluster_ld(cluster_addr(&s_m[q], lane));
          cl = cluster_ld(cluster_addr(&s_l[q], lane));
        }
        const float top = warp_max(cm), f = weight(cm, top);
        const float sum = warp_sum(cm == -INFINITY ? cl : f * cl);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        const int c = lane & (CH - 1);
        const uint32_t own = smem_u32(reinterpret_cast<float4*>(ring) + q * CH + (c ^ (q & (CH - 1))));
        // from the next CTA on (all starting at CTA 0 would queue there), all loads
        // in flight together; the order is the row's own, so results repeat
        float4 v[kMaxSplit];
#pragma unroll
        for (int k = 0; k < kMaxSplit; ++k)
          if (k < split) v[k] = cluster_ld4(cluster_map(own, (part + k) % split));
#pragma unroll
        for (int k = 0; k < kMaxSplit; ++k) {
          const float fk = __shfl_sync(0xffffffffu, f, (part + k) % split);
          if (k < split && fk != 0.f) {  // (a CTA without keys has written no O)
            acc.x += fk * v[k].x;
            acc.y += fk * v[k].y;
            acc.z += fk * v[k].z;
            acc.w += fk * v[k].w;
          }
        }
        const int i = row0 + q, t = sh.by_rep.quot(i), h = hk * rep + i - t * rep;
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        const bool fin = isfinite(acc.x * inv) && isfinite(acc.y * inv) && isfinite(acc.z * inv) && isfinite(acc.w * inv);
        uint16_t* dst = static_cast<uint16_t*>(a.out) + b * a.os[0] + t * a.os[1] + h * a.os[2] + c * 4;
        if (lane < CH)
          *reinterpret_cast<uint2*>(dst) =
              make_uint2(pack2<F16>(acc.x * inv, acc.y * inv), pack2<F16>(acc.z * inv, acc.w * inv));
        if (lane == 0 && a.lse)
          a.lse[((long long)b * a.Tq + t) * a.Hq + h] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
        if (__any_sync(0xffffffffu, !fin) && !__any_sync(0xffffffffu, s_fail)) {
          __syncwarp();  // (its stores come after those above)
          exact_row<HD, F16>(a, b, t, h, n, ql, lane);
        }
      }
      cluster_barrier();  // nobody leaves while its shared memory may still be read
    }
  }
  fence_before();
  __syncthreads();
  if (tid == 0 && s_fail) {
    // the copies in flight still land before anybody leaves (here: a wait may
    // give up after the copying has ended)
    for (int q = max(0, s_loaded - NST); q < s_loaded; ++q) mbar_wait(&bar.full[q % NST], (q / NST) & 1, kSpin);
    if (a.err) atomicOr(a.err, RL_DEVERR_TIMEOUT);
  }
  if (warp == 9) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
}

// The map of Q's rows (see RowsShape); false: not of a form that a box of 128
// rows fits, and the threads load them.
bool make_q_map(CUtensorMap* map, const AttnOpArgs& a, bool prefix) {
  const int rep = a.Hq / a.Hkv;
  if (a.q_f32 || 128 % rep) return false;
  const int seqs = prefix ? 1 : a.B, rows = prefix ? a.B : a.Tq;
  // (an axis of extent 1 takes any stride)
  const long long st[3] = {a.Hq > 1 ? a.qs[2] : a.hd, rows > 1 ? (prefix ? a.qs[0] : a.qs[1]) : a.hd, seqs > 1 ? a.qs[0] : a.hd};
  for (long long x : st)
    if (x == 0 || x >= (1ll << 39)) return false;
  const cuuint64_t dims[5] = {64, (cuuint64_t)a.Hq, (cuuint64_t)rows, (cuuint64_t)(a.hd / 64), (cuuint64_t)seqs};
  const cuuint64_t strides[4] = {(cuuint64_t)st[0] * 2, (cuuint64_t)st[1] * 2, 128, (cuuint64_t)st[2] * 2};
  const cuuint32_t box[5] = {64, (cuuint32_t)rep, (cuuint32_t)(128 / rep), (cuuint32_t)(a.hd / 64), 1};
  const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  return tensor_map_encoder()(map, a.f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5,
                              const_cast<void*>(a.q), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int HD, bool F16, bool PREFIX>
cudaError_t launch(const AttnOpArgs& a, cudaStream_t s) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = device_sm_count(dev, &sms);
  if (e != cudaSuccess) return e;
  auto kern = k_attn_rows_tc<HD, F16, PREFIX>;
  const int* clusters = nullptr;  // that fit the GPU at once, by their CTAs (fixed once set)
  {
    static std::mutex mu;
    static bool done[kOpDevices] = {};
    static int room[kOpDevices][kMaxSplit + 1];
    std::lock_guard<std::mutex> lock(mu);
    if (!done[dev]) {
      e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem<HD>);
      for (int c = 1; c <= kMaxSplit && !PREFIX && e == cudaSuccess; ++c) {
        cudaLaunchConfig_t q = {};
        q.gridDim = dim3(c);
        q.blockDim = dim3(kThreads);
        q.dynamicSmemBytes = kSmem<HD>;
        cudaLaunchAttribute at[1];
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = c;
        at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
        q.attrs = at;
        q.numAttrs = 1;
        e = cudaOccupancyMaxActiveClusters(&room[dev][c], kern, &q);
      }
      if (e != cudaSuccess) return e;
      done[dev] = true;
    }
    clusters = room[dev];
  }
  KvMaps maps;
  const bool got = PREFIX ? make_kv_maps(&maps, a.pre, a.f16 != 0, 1, a.Hkv, HD, a.P, kKeys)
                          : make_kv_maps(&maps, a.kv, a.f16 != 0, a.B, a.Hkv, HD, a.cap, kKeys);
  if (!got) return cudaErrorInvalidValue;
  const int rep = a.Hq / a.Hkv;
  const long long rows = (long long)(PREFIX ? a.B : a.Tq) * rep;
  const int tiles = (int)((rows + kRowsCta - 1) / kRowsCta);
  const long long ctas = (long long)tiles * a.Hkv * (PREFIX ? 1 : a.B);
  int split = 1;
  if (PREFIX) {
    split = prefix_split(a.B, rep, a.Hkv, a.P);
  } else {
    // the count with the least time by this model (clocks, measured): waves of
    // clusters, each a CTA's start and end, its tiles of 128 keys, a cluster's join
    const long long keys = min((long long)a.cap, (long long)a.window + min(a.Tq, kRowsCta / rep + 2) + a.sinks);
    const long long nt = (keys + kKeys - 1) / kKeys;
    double least = 0;
    for (int c = 1; c <= kMaxSplit && c <= nt; ++c) {
      if (clusters[c] < 1) continue;
      const double t = (double)((ctas + clusters[c] - 1) / clusters[c]) *
                       (10000 + (double)((nt + c - 1) / c) * (rows > 128 ? 3400 : 2500) + (c > 1 ? 6000 : 0));
      if (c == 1 || t < least) {
        split = c;
        least = t;
      }
    }
  }
  if (ctas * split >= (1ll << 31) - 4096) return cudaErrorInvalidValue;  // (a cluster some SMs ahead has a number too)
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(ctas * split));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem<HD>;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = PREFIX ? 1 : split;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  RowsShape sh;
  CUtensorMap q_map = {};
  const long long polls = g_wait_polls.load();
  sh.polls = polls < 0 ? kSpin : (int)min(polls, (long long)kSpin);
  sh.split = split;
  sh.tiles = tiles;
  sh.q_tma = make_q_map(&q_map, a, PREFIX);
  sh.ahead = PREFIX ? 0 : clusters[split];
  sh.apart = PREFIX && prefix_apart(a.B, rep, a.Hkv);
  sh.by_split = FastDiv(split);
  sh.by_heads = FastDiv(a.Hkv);
  sh.by_group = FastDiv(PREFIX ? a.Hkv : a.Hkv * a.B);
  sh.by_rep = FastDiv(rep);
  return cudaLaunchKernelEx(&cfg, kern, maps, q_map, a, sh);
}

template <bool PREFIX>
cudaError_t launch_any(const AttnOpArgs& a, cudaStream_t s) {
  if (a.hd == 64) return a.f16 ? launch<64, true, PREFIX>(a, s) : launch<64, false, PREFIX>(a, s);
  return a.f16 ? launch<128, true, PREFIX>(a, s) : launch<128, false, PREFIX>(a, s);
}

}  // namespace

// Keys' splits of a prefix: the count with the least time by this model (clocks,
// measured): a CTA's start and end, its tiles of 128 keys (two row tiles, or
// one), and the workspace traffic of a part.  152 SMs are planned for, so that
// the workspace's size does not depend on the device.
// CTAs of the prefix's products, at most, when the own keys' run beside them
// (256 sequences behind 32768 tokens, 32 heads, 8 KV heads, head_dim
// 128, own keys up to 2000: 64 CTAs 249 us, 96 221, 128 255, 152 254; one after
// the other, on all SMs, 274).  Each (row tile, KV head) gets the whole number of
// parts below that, so the CTAs there are vary: at these heads 96 for 80 to 256
// sequences, 80 for 320, 64 for 512, 128 for 1024 (one part each).
constexpr int kApartCtas = 100;
// More own-key CTAs than four an SM, of which three run at once (8 KV heads, head_dim 128, joined apart
// against in place: 32 sequences behind 8192, up to 1024 of their own, 33.1 us
// against 30.1, 64 45.4 against 46.3, 128 65.2 against 70.2; behind 1024, up to
// 256, 14.5 against 12.2, 20.2 against 21.0, 29.0 against 29.6; called one by one
// the third launch costs 2 us more).  It knows neither the prefix's length nor
// the capacity.  With a long prefix and few own keys in place is faster, the
// more the fewer CTAs the constant above leaves (behind 32768, up to 16 of their
// own, apart against in place: 80 sequences 88 us against 70, 128 88 against 78,
// 256 165 against 151, 512 463 against 290; up to 2000: 98 against 105, 127
// against 151, 226 against 278, 473 against 520; behind 8192, up to 512: 36
// against 39, 50 against 54, 83 against 90, 139 against 161).
bool prefix_apart(int B, int rep, int Hkv) { return (long long)B * Hkv * ((rep + 15) / 16) > 4 * 152; }

int prefix_split(int B, int rep, int Hkv, int P) {
  const long long rows = (long long)B * rep, tiles = (rows + kRowsCta - 1) / kRowsCta, items = tiles * Hkv;
  const long long nt = ((long long)P + kKeys - 1) / kKeys;
  if (prefix_apart(B, rep, Hkv))  // the own keys run beside it on the other SMs
    return (int)max(1ll, min(min(kApartCtas / items, nt), (long long)kMaxPrefixSplit));
  const double tile = rows > 128 ? 3400 : 2500;
  const double part = 0.5 * attn::prefix_rows((int)tiles, rows);
  int best = 1;
  double least = 0;
  for (int s = 1; s <= kMaxPrefixSplit && s <= nt; ++s) {
    const double t = (double)((items * s + 151) / 152) * (10000 + (double)((nt + s - 1) / s) * tile) + part * items * s;
    if (s == 1 || t < least) {
      best = s;
      least = t;
    }
  }
  return best;
}

size_t prefix_ws_bytes(int B, int rep, int Hkv, int hd, int P) {
  const long long rows = (long long)B * rep;
  const int tiles = (int)((rows + kRowsCta - 1) / kRowsCta);
  const int split = P > 0 ? prefix_split(B, rep, Hkv, P) : 1;
  return (size_t)tiles * Hkv * (split + prefix_apart(B, rep, Hkv)) * attn::prefix_rows(tiles, rows) * (hd + 2) * sizeof(float);
}

cudaError_t launch_attn_rows_tc(const AttnOpArgs& a, bool prefix, cudaStream_t s) {
  return prefix ? launch_any<true>(a, s) : launch_any<false>(a, s);
}

}  // namespace river

extern "C" rl_status rl_debug_limit_waits(int64_t polls) {
  river::g_wait_polls.store(polls);
  return RL_OK;
}
