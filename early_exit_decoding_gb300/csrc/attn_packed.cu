// Causal attention of packed prompts (rl_packed_attention): the rows of
// attn_rows_tc.cu, whose CTAs find their sequence and row tile themselves
// (row_tile: longest first, so the last CTAs to start have the fewest keys).
//
// Tensor cores bound it as they do one prompt: two prompts of 8192 and 5001
// tokens, 32 heads, 8 KV heads, head_dim 128: 600 us, 1.26 PFLOP/s, 0.65 of the
// measured bf16 rate; 12 of 37 to 2999: 325 us, 0.49, as a CTA's start and end
// weigh more on fewer key tiles.  17 of 1 to 97 tokens: 16 us, one tile's chain.
#include <string.h>

#include "kv4.cuh"

namespace river {

cudaError_t launch_packed_attention(const PackedArgs& p, cudaStream_t s) {
  AttnOpArgs o;
  memset(&o, 0, sizeof(o));
  o.q = p.q;
  o.out = p.out;
  o.lse = p.lse;
  o.kv.k = p.k;
  o.kv.v = p.v;
  for (int i = 0; i < 2; ++i) {
    o.qs[1 + i] = p.qs[i];
    o.os[1 + i] = p.os[i];
    o.kv.ks[2 - i] = p.ks[i];
    o.kv.vs[2 - i] = p.vs[i];
  }
  o.f16 = p.f16;
  o.B = p.B;
  o.Tq = p.max_rows;
  o.cap = p.N;
  o.Hq = p.Hq;
  o.Hkv = p.Hkv;
  o.hd = p.hd;
  o.window = 1 << 30;  // (every key)
  o.scale = p.scale;
  o.start = p.start;
  o.err = p.err;
  return launch_attn_rows_tc(o, false, s);
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
