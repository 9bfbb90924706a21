// Attention over the paged cache held in 4 bits (rl_kv4_attention): single
// tokens and drafts.
//
// Simplest form: a warp a row and query head, one key at a time, running maximum
// and sum; a key's value is m + s c in fp32.
#include <float.h>
#include <math.h>

#include "kv4.cuh"

namespace river {

namespace {

using namespace dev;
using namespace attn;

template <int HD, bool F16>
__global__ void __launch_bounds__(256) k_kv4_attn(const __grid_constant__ PackedArgs a, const __grid_constant__ Kv4Args c) {
  constexpr int NB = HD / 64;  // bytes of codes a lane takes
  const int lane = threadIdx.x & 31;
  check_start(a);
  const long long w = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int r = (int)(w / a.Hq), h = (int)(w - (long long)r * a.Hq);
  if (r >= a.N) return;
  const int b = seq_of_row(a, r, lane);
  if (b < 0) return;
  const Span sp = seq_span(a, b, h == 0 && lane == 0);
  if (r - sp.first >= sp.n) return;
  const long long cap = (long long)c.width << c.page_log;
  const int len = __ldg(a.kv_len + b);
  if (a.err && h == 0 && lane == 0 && (len < 0 || len > cap)) atomicOr(a.err, RL_DEVERR_CAPACITY);
  const int n = (int)max(0ll, min((long long)len, cap)), end = n - sp.all + (r - sp.first) + 1, hk = h / (a.Hq / a.Hkv);
  float q[2 * NB], o[2 * NB] = {}, m = -INFINITY, l = 0.f;
  const uint16_t* qp = static_cast<const uint16_t*>(a.q) + r * a.qs[0] + h * a.qs[1] + 2 * NB * lane;
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    const float2 f = unpack2<F16>(*reinterpret_cast<const uint32_t*>(qp + 2 * i));
    q[2 * i] = f.x;
    q[2 * i + 1] = f.y;
  }
  for (int j = 0; j < end; ++j) {
    const long long page = max(page_at(a, c, b, j >> c.page_log), 0), at = page_row(c, hk, j & ((1 << c.page_log) - 1));
    const unsigned char* kc = c.kc + page * c.kc_step + at * (HD / 2) + NB * lane;
    const unsigned char* vc = c.vc + page * c.vc_step + at * (HD / 2) + NB * lane;
    const float2 km = unpack2<F16>(c.km[page * c.km_step + at]), vm = unpack2<F16>(c.vm[page * c.vm_step + at]);
    float d = 0.f;
#pragma unroll
    for (int i = 0; i < NB; ++i)
      d += q[2 * i] * (km.y + km.x * (float)(kc[i] & 15)) + q[2 * i + 1] * (km.y + km.x * (float)(kc[i] >> 4));
    d = warp_sum(d) * a.scale;
    const float mn = fmaxf(m, d), mu = mn == -INFINITY ? 0.f : mn, f = __expf(m - mu), e = __expf(d - mu);
    l = l * f + e;
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      o[2 * i] = o[2 * i] * f + e * (vm.y + vm.x * (float)(vc[i] & 15));
      o[2 * i + 1] = o[2 * i + 1] * f + e * (vm.y + vm.x * (float)(vc[i] >> 4));
    }
    m = mn;
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  uint16_t* op = static_cast<uint16_t*>(a.out) + r * a.os[0] + h * a.os[1] + 2 * NB * lane;
#pragma unroll
  for (int i = 0; i < NB; ++i) *reinterpret_cast<uint32_t*>(op + 2 * i) = pack2<F16>(o[2 * i] * inv, o[2 * i + 1] * inv);
  if (lane == 0 && a.lse) a.lse[(long long)r * a.Hq + h] = l == 0.f ? -INFINITY : m + logf(l);
}

}  // namespace

cudaError_t launch_kv4_attention(const PackedArgs& p, const Kv4Args& c, cudaStream_t s) {
  const unsigned grid = (unsigned)(((long long)p.N * p.Hq + 7) / 8);
  if (p.hd == 64)
    p.f16 ? k_kv4_attn<64, true><<<grid, 256, 0, s>>>(p, c) : k_kv4_attn<64, false><<<grid, 256, 0, s>>>(p, c);
  else
    p.f16 ? k_kv4_attn<128, true><<<grid, 256, 0, s>>>(p, c) : k_kv4_attn<128, false><<<grid, 256, 0, s>>>(p, c);
  return cudaGetLastError();
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
