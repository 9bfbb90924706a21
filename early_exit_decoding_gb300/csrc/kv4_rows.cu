// Rows into and out of the paged cache held in 4 bits: rl_kv4_append (position
// rotation, quantisation, scatter to the pages) and rl_kv4_read (the values of
// rows), and the checks that the packed operators share.
//
// A row of head_dim values is one group: m = min x, s = (max x - m) / 15 in the
// cache's type, c = rint((x - m) / s), value m + s c.  m is a value of the row
// and so exact; s is rounded before the codes are taken, which costs the
// largest values half a step of s at most (2^-9 of the range in bf16).
//
// What bounds it: instructions, then HBM.  8169 rows of 32 + 2 x 8 heads of 128:
// append 42 us for 170 MB (0.6 of a measured copy; 26 M warp instructions, a
// third of them the rotation's conversions, a third the codes), reading back 16
// (16-byte stores 32 bytes apart: half of every sector an instruction).
// (Packed fp32 products and sums would halve the rotation's, but written as they
// are they came out fused, one rounding short, and codes must not depend on that;
// sums as fma by a 1 that the compiler cannot see have not been tried.)  A decode
// step's rows: 7 us and 6, launches and chains of loads.
#include <float.h>
#include <math.h>
#include <stdio.h>
#include <string.h>

#include "kv4.cuh"

namespace river {

namespace {

using namespace dev;
using namespace attn;

constexpr int kThreads = 256;
constexpr int kAppendCtas = 4;  // of an SM (8192 rows of 48 heads: three 70 us with the reading back, four 61, five 63)
constexpr float kLeastStep = 7.888609052210118e-31f;  // 2^-100

// Maximum and minimum that a NaN survives.
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float min_nan(float a, float b) {
  float d;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// Codes rint((f - mn) / s) of 16 values (s > 0): lo of the first eight, hi of the
// others.  f - mn times 1 / s is off the quotient by less than 2^-18 (it is below
// 16, or 22 where s is a denormal number of fp16), so it rounds alike unless that
// near to half a step, ties among them: those are divided.
__device__ __forceinline__ void codes_of(const float (&f)[16], float mn, float s, uint32_t* lo, uint32_t* hi) {
  const float big = 12582912.f;  // 1.5 2^23: its sums are whole numbers
  const float inv = __fdiv_rn(1.f, s);
  uint32_t w[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {  // (four at a time: some tie is in two thirds of a warp's 512 bf16 values)
    float c[4], far = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float t = __fmul_rn(__fsub_rn(f[4 * q + e], mn), inv);
      c[e] = __fsub_rn(__fadd_rn(t, big), big);
      far = fmaxf(far, fabsf(__fsub_rn(t, c[e])));
    }
    if (!(far < 0.5f - 3.814697265625e-6f)) {
#pragma unroll
      for (int e = 0; e < 4; ++e) c[e] = rintf(__fdiv_rn(__fsub_rn(f[4 * q + e], mn), s));
    }
    // four codes as the digits of a number below 2^16 (NaN gives 0: the row's s or m says so)
    float d = 0.f;
#pragma unroll
    for (int e = 3; e >= 0; --e) d = fmaf(d, 16.f, fminf(fmaxf(c[e], 0.f), 15.f));
    w[q] = __float_as_uint(d + big) & 0xffffu;
  }
  *lo = w[0] | w[1] << 16;
  *hi = w[2] | w[3] << 16;
}

// Sequence (-1: none) and position of packed row r.
__device__ __forceinline__ long long row_place(const PackedArgs& a, int r, int lane, int* seq) {
  const int b = seq_of_row(a, r, lane);
  *seq = b;
  if (b < 0) return -1;
  const int end = a.start ? min(__ldg(a.start + b + 1), a.N) : r + 1;
  return (long long)__ldg(a.kv_len + b) - end + r;
}

// A warp takes `iters` times 32 / L heads of one row, L = HD / 16 lanes a head:
// lane i of them dims 8 i .. 8 i + 7 and the same from HD / 2 on, which are each
// other's rotation partners, so a row's angles are read once for all its heads.
template <int HD, bool F16>
__global__ void __launch_bounds__(kThreads, kAppendCtas)
    k_kv4_append(const __grid_constant__ PackedArgs a, const __grid_constant__ Kv4Args c, const float2* __restrict__ rope,
                 int rope_len, int nq, int iters, FastDiv by_chunks) {
  constexpr int L = HD / 16, RPW = 32 / L;
  const int lane = threadIdx.x & 31, i = lane & (L - 1);
  const int w = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  check_start(a);
  const int r = by_chunks.quot(w);
  if (r >= a.N) return;
  int b;
  const long long pos = row_place(a, r, lane, &b);
  if (b < 0) return;
  if (pos < 0 || pos >= ((long long)c.width << c.page_log) || (rope && pos >= rope_len)) {
    if (a.err && lane == 0) atomicOr(a.err, RL_DEVERR_CAPACITY);
    return;
  }
  const int page = page_at(a, c, b, (int)(pos >> c.page_log)), prow = (int)pos & ((1 << c.page_log) - 1);
  if (page < 0) return;
  float4 cs[4];  // (cos, sin) of two pairs each
  if (rope) {
    const float4* t = reinterpret_cast<const float4*>(rope + pos * (HD / 2) + 8 * i);
#pragma unroll
    for (int e = 0; e < 4; ++e) cs[e] = __ldg(t + e);
  }
  const int total = nq + 2 * a.Hkv;
  int slot = (w - r * by_chunks.d) * iters * RPW + lane / L;
  for (int it = 0; it < iters; ++it, slot += RPW) {
    const bool live = slot < total;
    const int kind = slot < nq ? 0 : slot < nq + a.Hkv ? 1 : 2, h = slot - (kind == 0 ? 0 : kind == 1 ? nq : nq + a.Hkv);
    const void* base = kind == 0 ? a.q : kind == 1 ? a.k : a.v;
    const long long* st = kind == 0 ? a.qs : kind == 1 ? a.ks : a.vs;
    uint4 lo = make_uint4(0, 0, 0, 0), hi = lo;
    if (live) {
      const uint16_t* x = static_cast<const uint16_t*>(base) + r * st[0] + h * st[1] + 8 * i;
      lo = *reinterpret_cast<const uint4*>(x);  // (q may be written in its place)
      hi = *reinterpret_cast<const uint4*>(x + HD / 2);
    }
    uint32_t xl[4] = {lo.x, lo.y, lo.z, lo.w}, xh[4] = {hi.x, hi.y, hi.z, hi.w};
    if (rope && kind != 2) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {  // (each product and sum rounded once, so that codes do not depend on contraction)
        const float2 u = unpack2<F16>(xl[e]), v = unpack2<F16>(xh[e]);
        const float4 t = cs[e];
        xl[e] = pack2<F16>(__fsub_rn(__fmul_rn(u.x, t.x), __fmul_rn(v.x, t.y)), __fsub_rn(__fmul_rn(u.y, t.z), __fmul_rn(v.y, t.w)));
        xh[e] = pack2<F16>(__fadd_rn(__fmul_rn(v.x, t.x), __fmul_rn(u.x, t.y)), __fadd_rn(__fmul_rn(v.y, t.z), __fmul_rn(u.y, t.w)));
      }
    }
    if (live && kind == 0) {
      uint16_t* o = static_cast<uint16_t*>(a.out) + r * a.os[0] + h * a.os[1] + 8 * i;
      *reinterpret_cast<uint4*>(o) = make_uint4(xl[0], xl[1], xl[2], xl[3]);
      *reinterpret_cast<uint4*>(o + HD / 2) = make_uint4(xh[0], xh[1], xh[2], xh[3]);
    }
    if (!__any_sync(0xffffffffu, live && kind != 0)) continue;
    float f[16];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 u = unpack2<F16>(xl[e]), v = unpack2<F16>(xh[e]);
      f[2 * e] = u.x;
      f[2 * e + 1] = u.y;
      f[8 + 2 * e] = v.x;
      f[8 + 2 * e + 1] = v.y;
    }
    float mn = f[0], mx = f[0];
#pragma unroll
    for (int e = 1; e < 16; ++e) {
      mn = min_nan(mn, f[e]);
      mx = max_nan(mx, f[e]);
    }
#pragma unroll
    for (int d = 1; d < L; d <<= 1) {
      mn = min_nan(mn, __shfl_xor_sync(0xffffffffu, mn, d));
      mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, d));
    }
    float s = unpack2<F16>(pack2<F16>(__fdiv_rn(__fsub_rn(mx, mn), 15.f), 0.f)).x;
    if (s < kLeastStep) s = 0.f;
    uint32_t cl = 0, ch = 0;
    if (s != 0.f) codes_of(f, mn, s, &cl, &ch);
    if (live && kind != 0) {
      const long long at = page_row(c, h, prow);
      unsigned char* codes = (kind == 1 ? c.kc + page * c.kc_step : c.vc + page * c.vc_step) + at * (HD / 2) + 4 * i;
      *reinterpret_cast<uint32_t*>(codes) = cl;
      *reinterpret_cast<uint32_t*>(codes + HD / 4) = ch;
      if (i == 0) (kind == 1 ? c.km + page * c.km_step : c.vm + page * c.vm_step)[at] = pack2<F16>(s, mn);
    }
  }
}

// A warp takes `iters` times 32 / L rows of (k, v) x heads, a lane 16 values.
template <int HD, bool F16>
__global__ void __launch_bounds__(kThreads)
    k_kv4_read(const __grid_constant__ PackedArgs a, const __grid_constant__ Kv4Args c, uint16_t* __restrict__ k,
               uint16_t* __restrict__ v, int iters, FastDiv by_chunks) {
  constexpr int L = HD / 16, RPW = 32 / L;
  const int lane = threadIdx.x & 31, i = lane & (L - 1);
  const int w = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  check_start(a);
  const int r = by_chunks.quot(w);
  if (r >= a.N) return;
  int b;
  const long long pos = row_place(a, r, lane, &b);
  if (b < 0) return;
  if (pos < 0 || pos >= ((long long)c.width << c.page_log)) {
    if (a.err && lane == 0) atomicOr(a.err, RL_DEVERR_CAPACITY);
    return;
  }
  const int page = max(page_at(a, c, b, (int)(pos >> c.page_log)), 0), prow = (int)pos & ((1 << c.page_log) - 1);
  int slot = (w - r * by_chunks.d) * iters * RPW + lane / L;
  for (int it = 0; it < iters && slot < 2 * a.Hkv; ++it, slot += RPW) {
    const bool val = slot >= a.Hkv;
    const int h = val ? slot - a.Hkv : slot;
    const long long at = page_row(c, h, prow);
    const uint2 codes = __ldg(reinterpret_cast<const uint2*>((val ? c.vc + page * c.vc_step : c.kc + page * c.kc_step) + at * (HD / 2)) + i);
    const float2 sm = unpack2<F16>(__ldg((val ? c.vm + page * c.vm_step : c.km + page * c.km_step) + at));
    uint32_t o[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      // a code's float: 2^23 + c less 2^23; s c is exact (15 bits), so one rounding of the sum
      const uint32_t x = (e < 4 ? codes.x : codes.y) >> (8 * (e & 3));
      const float c0 = __uint_as_float((x & 15) | 0x4b000000u) - 8388608.f, c1 = __uint_as_float((x >> 4 & 15) | 0x4b000000u) - 8388608.f;
      o[e] = pack2<F16>(fmaf(sm.x, c0, sm.y), fmaf(sm.x, c1, sm.y));
    }
    uint16_t* dst = (val ? v + r * a.vs[0] + h * a.vs[1] : k + r * a.ks[0] + h * a.ks[1]) + 16 * i;
    *reinterpret_cast<uint4*>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
    *reinterpret_cast<uint4*>(dst + 8) = make_uint4(o[4], o[5], o[6], o[7]);
  }
}

// A row's heads go to one warp where there are warps enough without, else to as
// many as there are groups of heads.
// (8192 rows of 48 heads of 128, with the reading back: 82 us with a group a
// warp, 68 with four, 61 with all twelve)
int chunk_iters(int groups, int rows, int sms) { return (long long)rows >= 16ll * sms ? groups : 1; }

// What a warp takes, and the blocks for all rows.
cudaError_t plan(int slots, int hd, int rows, int* iters, int* chunks, unsigned* grid) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = device_sm_count(dev, &sms);
  if (e != cudaSuccess) return e;
  const int rpw = 512 / hd, groups = (slots + rpw - 1) / rpw;
  *iters = chunk_iters(groups, rows, sms);
  *chunks = (groups + *iters - 1) / *iters;
  const long long warps = (long long)rows * *chunks;
  if (warps >= (1ll << 31) - kThreads) return cudaErrorInvalidValue;
  *grid = (unsigned)((warps + kThreads / 32 - 1) / (kThreads / 32));
  return cudaSuccess;
}

}  // namespace

rl_status op_error(const char* who, rl_status st, const char* what) {
  char msg[256];
  snprintf(msg, sizeof(msg), "%s: %s", who, what);
  return set_error(st, msg);
}
bool op_aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

rl_status check_packed(const char* who, const rl_packed_desc* p, int reads, int writes, PackedArgs* o) {
  if (!p) return op_error(who, RL_ERR_INVALID_ARG, "the descriptor is NULL");
  if (p->dtype != RL_DT_BF16 && p->dtype != RL_DT_F16)
    return op_error(who, RL_ERR_UNSUPPORTED, "dtype must be RL_DT_BF16 or RL_DT_F16");
  if (p->batch < 1 || p->rows < 1 || p->max_rows < 0 || p->n_kv_heads < 1 || p->n_q_heads < 1)
    return op_error(who, RL_ERR_INVALID_ARG, "batch, rows and heads must be >= 1, max_rows >= 0");
  if (p->batch > 1 << 16 || p->rows > 1 << 27 || (long long)p->rows * p->n_q_heads >= 1ll << 31 || p->n_kv_heads > 1 << 10)
    return op_error(who, RL_ERR_UNSUPPORTED, "batch must be at most 2^16, rows 2^27, rows * n_q_heads below 2^31, n_kv_heads at most 2^10");
  if (p->head_dim != 64 && p->head_dim != 128) return op_error(who, RL_ERR_UNSUPPORTED, "head_dim must be 64 or 128");
  if (p->n_q_heads % p->n_kv_heads) return op_error(who, RL_ERR_UNSUPPORTED, "n_q_heads must be a multiple of n_kv_heads");
  if (!(p->scale >= 0.f) || p->scale > 1e6f) return op_error(who, RL_ERR_INVALID_ARG, "scale must be in [0, 1e6]");
  memset(o, 0, sizeof(*o));
  const int64_t* from[4] = {p->q_stride, p->k_stride, p->v_stride, p->out_stride};
  long long* to[4] = {o->qs, o->ks, o->vs, o->os};
  for (int i = 0; i < 4; ++i) {
    if (!((reads | writes) >> i & 1)) continue;
    const int64_t heads = i == 0 || i == 3 ? p->n_q_heads : p->n_kv_heads, row = from[i][0], head = from[i][1];
    if (row < 0 || head < 0 || row % 8 || head % 8 || row >= 1ll << 39 || head >= 1ll << 39)
      return op_error(who, RL_ERR_UNSUPPORTED, "strides must be whole multiples of 16 bytes, below 2^39 elements");
    if (writes >> i & 1) {
      // from the smaller stride on, each axis steps over all that lies within it
      const bool rows_in = row <= head;
      const int64_t s0 = rows_in ? row : head, n0 = rows_in ? p->rows : heads, s1 = rows_in ? head : row, n1 = rows_in ? heads : p->rows;
      const double span = p->head_dim + (n0 > 1 ? (double)s0 * (double)(n0 - 1) : 0.0);
      if ((n0 > 1 && s0 < p->head_dim) || (n1 > 1 && (double)s1 < span))
        return op_error(who, RL_ERR_INVALID_ARG, "rows of an output overlap");
    }
    to[i][0] = row;
    to[i][1] = head;
  }
  o->f16 = p->dtype == RL_DT_F16;
  o->B = p->batch;
  o->N = p->rows;
  o->max_rows = p->max_rows > 0 && p->max_rows < p->rows ? p->max_rows : p->rows;
  o->Hq = p->n_q_heads;
  o->Hkv = p->n_kv_heads;
  o->hd = p->head_dim;
  o->scale = p->scale > 0.f ? p->scale : 1.f / sqrtf((float)p->head_dim);
  return RL_OK;
}

rl_status check_kv4(const char* who, const rl_kv4* c, const PackedArgs& p, Kv4Args* o) {
  if (!c) return op_error(who, RL_ERR_INVALID_ARG, "the cache is NULL");
  if (c->n_pages < 1 || c->table_width < 1) return op_error(who, RL_ERR_INVALID_ARG, "n_pages and table_width must be >= 1");
  int lg = 4;
  while (lg < 8 && (1 << lg) != c->page) ++lg;
  if (1 << lg != c->page) return op_error(who, RL_ERR_UNSUPPORTED, "page must be 16, 32, 64, 128 or 256");
  if (((long long)c->table_width << lg) > 1ll << 30) return op_error(who, RL_ERR_UNSUPPORTED, "table_width * page must be at most 2^30");
  if (!c->k_codes || !c->k_scale || !c->v_codes || !c->v_scale || !c->d_table)
    return op_error(who, RL_ERR_INVALID_ARG, "a buffer of the cache is NULL");
  if (!op_aligned16(c->k_codes) || !op_aligned16(c->k_scale) || !op_aligned16(c->v_codes) || !op_aligned16(c->v_scale) ||
      (reinterpret_cast<uintptr_t>(c->d_table) & 3))
    return op_error(who, RL_ERR_UNSUPPORTED, "the cache's buffers must start on 16-byte boundaries (the table on 4)");
  const int64_t rows = (int64_t)p.Hkv << lg;
  if (p.B > 1 && (c->table_stride < c->table_width || c->table_stride >= 1ll << 40))
    return op_error(who, RL_ERR_INVALID_ARG, "table_stride must be at least table_width, below 2^40");
  for (int i = 0; i < 2 && c->n_pages > 1; ++i) {
    if (c->code_stride[i] % 16 || c->scale_stride[i] % 8 || c->code_stride[i] >= 1ll << 31 || c->scale_stride[i] >= 1ll << 30)
      return op_error(who, RL_ERR_UNSUPPORTED, "page strides must be whole multiples of 16 bytes, below 2^31 bytes");
    if (c->code_stride[i] < rows * (p.hd / 2) || c->scale_stride[i] < rows * 2)
      return op_error(who, RL_ERR_INVALID_ARG, "pages overlap");
  }
  o->n_pages = c->n_pages;
  o->page_log = lg;
  o->kc = static_cast<unsigned char*>(c->k_codes);
  o->vc = static_cast<unsigned char*>(c->v_codes);
  o->km = static_cast<uint32_t*>(c->k_scale);
  o->vm = static_cast<uint32_t*>(c->v_scale);
  const bool many = c->n_pages > 1;  // (of one page no stride matters)
  o->kc_step = many ? c->code_stride[0] : 0;
  o->vc_step = many ? c->code_stride[1] : 0;
  o->km_step = many ? c->scale_stride[0] / 2 : 0;
  o->vm_step = many ? c->scale_stride[1] / 2 : 0;
  o->table = c->d_table;
  o->table_step = p.B > 1 ? c->table_stride : 0;
  o->width = c->table_width;
  return RL_OK;
}

cudaError_t launch_kv4_append(const PackedArgs& p, const Kv4Args& c, const float2* rope, int rope_len, cudaStream_t s) {
  const int nq = p.q ? p.Hq : 0;
  int iters, chunks;
  unsigned grid;
  const cudaError_t e = plan(nq + 2 * p.Hkv, p.hd, p.N, &iters, &chunks, &grid);
  if (e != cudaSuccess) return e;
  const FastDiv by(chunks);
  if (p.hd == 64)
    p.f16 ? k_kv4_append<64, true><<<grid, kThreads, 0, s>>>(p, c, rope, rope_len, nq, iters, by)
          : k_kv4_append<64, false><<<grid, kThreads, 0, s>>>(p, c, rope, rope_len, nq, iters, by);
  else
    p.f16 ? k_kv4_append<128, true><<<grid, kThreads, 0, s>>>(p, c, rope, rope_len, nq, iters, by)
          : k_kv4_append<128, false><<<grid, kThreads, 0, s>>>(p, c, rope, rope_len, nq, iters, by);
  return cudaGetLastError();
}

cudaError_t launch_kv4_read(const PackedArgs& p, const Kv4Args& c, void* k, void* v, cudaStream_t s) {
  int iters, chunks;
  unsigned grid;
  const cudaError_t e = plan(2 * p.Hkv, p.hd, p.N, &iters, &chunks, &grid);
  if (e != cudaSuccess) return e;
  const FastDiv by(chunks);
  uint16_t *ko = static_cast<uint16_t*>(k), *vo = static_cast<uint16_t*>(v);
  if (p.hd == 64)
    p.f16 ? k_kv4_read<64, true><<<grid, kThreads, 0, s>>>(p, c, ko, vo, iters, by)
          : k_kv4_read<64, false><<<grid, kThreads, 0, s>>>(p, c, ko, vo, iters, by);
  else
    p.f16 ? k_kv4_read<128, true><<<grid, kThreads, 0, s>>>(p, c, ko, vo, iters, by)
          : k_kv4_read<128, false><<<grid, kThreads, 0, s>>>(p, c, ko, vo, iters, by);
  return cudaGetLastError();
}

}  // namespace river

using namespace river;

extern "C" rl_status rl_kv4_append(const rl_kv4* c, const rl_packed_desc* p, const int32_t* d_start,
                                   const int32_t* d_kv_len, const void* d_q, const void* d_k, const void* d_v,
                                   const float* d_rope, int32_t rope_len, void* d_out, int32_t* d_err, rl_stream_t stream) {
  const char* who = "rl_kv4_append";
  PackedArgs a;
  Kv4Args k;
  rl_status st = check_packed(who, p, d_q ? kUsesQ | kUsesK | kUsesV : kUsesK | kUsesV, d_q ? kUsesOut : 0, &a);
  if (st == RL_OK) st = check_kv4(who, c, a, &k);
  if (st != RL_OK) return st;
  if (!d_kv_len || !d_k || !d_v || (d_q && !d_out) || (d_rope && rope_len < 1))
    return op_error(who, RL_ERR_INVALID_ARG, "NULL argument, or rope_len below 1");
  if (!d_start && p->rows != p->batch) return op_error(who, RL_ERR_INVALID_ARG, "rows must be batch without d_start");
  if (!op_aligned16(d_q) || !op_aligned16(d_k) || !op_aligned16(d_v) || (d_q && !op_aligned16(d_out)) || !op_aligned16(d_rope))
    return op_error(who, RL_ERR_UNSUPPORTED, "q, k, v, out and the rotation's table must start on 16-byte boundaries");
  if (d_q && (d_out == d_k || d_out == d_v)) return op_error(who, RL_ERR_INVALID_ARG, "out overlaps an input");
  if (d_q && d_out == d_q && (a.qs[0] != a.os[0] || a.qs[1] != a.os[1]))
    return op_error(who, RL_ERR_INVALID_ARG, "out in q's place must have q's strides");
  a.q = d_q;
  a.k = d_k;
  a.v = d_v;
  a.out = d_out;
  a.start = d_start;
  a.kv_len = d_kv_len;
  a.err = d_err;
  const cudaError_t e = launch_kv4_append(a, k, reinterpret_cast<const float2*>(d_rope), rope_len, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return set_error(RL_ERR_CUDA, cudaGetErrorString(e));
  return RL_OK;
}

extern "C" rl_status rl_kv4_read(const rl_kv4* c, const rl_packed_desc* p, const int32_t* d_start, const int32_t* d_kv_len,
                                 void* d_k, void* d_v, int32_t* d_err, rl_stream_t stream) {
  const char* who = "rl_kv4_read";
  PackedArgs a;
  Kv4Args k;
  rl_status st = check_packed(who, p, 0, kUsesK | kUsesV, &a);
  if (st == RL_OK) st = check_kv4(who, c, a, &k);
  if (st != RL_OK) return st;
  if (!d_kv_len || !d_k || !d_v || d_k == d_v) return op_error(who, RL_ERR_INVALID_ARG, "NULL argument, or k and v in one place");
  if (!d_start && p->rows != p->batch) return op_error(who, RL_ERR_INVALID_ARG, "rows must be batch without d_start");
  if (!op_aligned16(d_k) || !op_aligned16(d_v)) return op_error(who, RL_ERR_UNSUPPORTED, "k and v must start on 16-byte boundaries");
  a.start = d_start;
  a.kv_len = d_kv_len;
  a.err = d_err;
  const cudaError_t e = launch_kv4_read(a, k, d_k, d_v, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return set_error(RL_ERR_CUDA, cudaGetErrorString(e));
  return RL_OK;
}
