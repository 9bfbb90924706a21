// Causal attention of packed prompts (rl_packed_attention).
//
// Simplest form: a warp a row and query head, one key at a time.
#include <float.h>
#include <math.h>

#include "kv4.cuh"

namespace river {

namespace {

using namespace dev;
using namespace attn;

template <int HD, bool F16>
__global__ void __launch_bounds__(256) k_packed(const __grid_constant__ PackedArgs a) {
  const int lane = threadIdx.x & 31;
  check_start(a);
  const long long w = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int r = (int)(w / a.Hq), h = (int)(w - (long long)r * a.Hq);
  if (r >= a.N) return;
  const int b = seq_of_row(a, r, lane);
  if (b < 0) return;
  const Span sp = seq_span(a, b, h == 0 && lane == 0);
  if (r - sp.first >= sp.n) return;
  AttnOpArgs o = {};
  o.q = a.q;
  o.out = a.out;
  o.lse = a.lse;
  o.Tq = a.N;
  o.Hq = a.Hq;
  for (int i = 0; i < 2; ++i) {
    o.qs[i + 1] = a.qs[i];
    o.os[i + 1] = a.os[i];
  }
  const KeySrc s{a.k, a.v, {0, a.ks[1], a.ks[0]}, {0, a.vs[1], a.vs[0]}};
  RowAcc<HD, F16> acc;
  acc.load_q(o, 0, r, h, lane);
  acc.keys(s, 0, h / (a.Hq / a.Hkv), sp.first, r + 1, a.scale, lane);
  acc.store(o, 0, r, h, lane);
}

}  // namespace

cudaError_t launch_packed_attention(const PackedArgs& p, cudaStream_t s) {
  const unsigned grid = (unsigned)(((long long)p.N * p.Hq + 7) / 8);
  if (p.hd == 64)
    p.f16 ? k_packed<64, true><<<grid, 256, 0, s>>>(p) : k_packed<64, false><<<grid, 256, 0, s>>>(p);
  else
    p.f16 ? k_packed<128, true><<<grid, 256, 0, s>>>(p) : k_packed<128, false><<<grid, 256, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace river

using namespace river;

extern "C" rl_status rl_packed_attention(const rl_packed_desc* p, const void* d_q, const void* d_k, const void* d_v,
                                         const int32_t* d_start, void* d_out, float* d_lse, int32_t* d_err, rl_stream_t stream) {
  const char* who = "rl_packed_attention";
  PackedArgs a;
  const rl_status st = check_packed(who, p, kUsesQ | kUsesK | kUsesV, kUsesOut, &a);
  if (st != RL_OK) return st;
  if (!d_q || !d_k || !d_v || !d_start || !d_out) return op_error(who, RL_ERR_INVALID_ARG, "NULL argument");
  if (p->rows > 1 && (a.ks[0] == 0 || a.vs[0] == 0)) return op_error(who, RL_ERR_UNSUPPORTED, "k and v row strides must not be 0");
  if (!op_aligned16(d_q) || !op_aligned16(d_k) || !op_aligned16(d_v) || !op_aligned16(d_out))
    return op_error(who, RL_ERR_UNSUPPORTED, "q, k, v and out must start on 16-byte boundaries");
  if (d_out == d_q || d_out == d_k || d_out == d_v) return op_error(who, RL_ERR_INVALID_ARG, "out overlaps an input");
  a.q = d_q;
  a.k = d_k;
  a.v = d_v;
  a.start = d_start;
  a.out = d_out;
  a.lse = d_lse;
  a.err = d_err;
  const cudaError_t e = launch_packed_attention(a, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return set_error(RL_ERR_CUDA, cudaGetErrorString(e));
  return RL_OK;
}
