// Stand-alone attention operators over caller-owned caches: sliding window
// with sinks (rl_window_attention) and a batch behind one shared prefix
// (rl_shared_prefix_attention).
//
// For a query row at position p:  out = sum_j w_j v_j / sum_j w_j with
// w_j = exp(scale q.k_j - m) over the keys j it sees and m their largest
// score;  lse = m + ln sum_j w_j.  Running maximum and sum, one pass.
// Few query rows go to attn_decode.cu, many to attn_rows_tc.cu.
#include <float.h>
#include <math.h>
#include <stdio.h>
#include <string.h>

#include <algorithm>

#include "attn_ops.cuh"

namespace river {

using namespace attn;

cudaError_t launch_window_attention(const AttnOpArgs& a, cudaStream_t s) {
  // up to 16 rows of a KV head (one m16 tile) are the few-row kernel's; with more
  // it would read the keys once a tile (window 2048, 8 KV heads, head_dim 128;
  // few-row against tensor-core kernel: 8 sequences of 4 rows 16.3 us against
  // 19.7, 16 rows 19.4 against 20.9, 20 rows 28.2 against 22.3, 64 rows 45.4
  // against 24.7; 64 sequences of 4 rows 96 against 114, 20 rows 134 against 125)
  if ((long long)a.Tq * (a.Hq / a.Hkv) <= 16) return launch_attn_decode(a, false, s);
  return launch_attn_rows_tc(a, false, s);
}

size_t shared_prefix_ws_bytes(int B, int Hq, int Hkv, int hd, int P) { return prefix_ws_bytes(B, Hq / Hkv, Hkv, hd, P); }

// The prefix for all rows first, then each sequence's own keys; the second
// kernel starts beside the first and takes the prefix's part at its end, or
// (many sequences) leaves its own part to a third that joins them.
cudaError_t launch_shared_prefix_attention(const AttnOpArgs& a, cudaStream_t s) {
  if (a.P > 0) {
    const cudaError_t e = launch_attn_rows_tc(a, true, s);
    if (e != cudaSuccess) return e;
  }
  const cudaError_t e = launch_attn_decode(a, a.P > 0, s);
  if (e != cudaSuccess || a.P == 0 || !prefix_apart(a.B, a.Hq / a.Hkv, a.Hkv)) return e;
  return launch_prefix_join(a, s);
}

}  // namespace river

using namespace river;

namespace {

constexpr int kMaxTokens = 1 << 30;  // of one source: key numbers a tile further stay in 31 bits

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

bool strides_ok(const int64_t* st, int n, int es, int64_t most) {
  for (int i = 0; i < n; ++i)
    if (st[i] < 0 || st[i] * es % 16 != 0 || st[i] >= most) return false;
  return true;
}

// Whether the rows of `row` elements at these strides (extents n) are apart:
// from the smallest stride on, each axis steps over all that lies within it.
bool rows_apart(const int64_t* st, const int64_t* n, int row) {
  int order[3] = {0, 1, 2};
  std::sort(order, order + 3, [&](int x, int y) { return st[x] < st[y]; });
  double span = row;
  for (int i : order) {
    if (n[i] == 1) continue;
    if ((double)st[i] < span) return false;
    span += (double)st[i] * (double)(n[i] - 1);
  }
  return true;
}

// The checks the two operators share; fills `o` from the descriptor.
rl_status check_desc(const char* who, const rl_attn_desc* a, AttnOpArgs* o) {
  auto bad = [&](rl_status st, const char* what) {
    char msg[256];
    snprintf(msg, sizeof(msg), "%s: %s", who, what);
    return set_error(st, msg);
  };
  if (!a) return bad(RL_ERR_INVALID_ARG, "the descriptor is NULL");
  if (a->kv_dtype != RL_DT_BF16 && a->kv_dtype != RL_DT_F16)
    return bad(RL_ERR_UNSUPPORTED, "kv_dtype must be RL_DT_BF16 or RL_DT_F16");
  if (a->q_dtype != a->kv_dtype && a->q_dtype != RL_DT_F32)
    return bad(RL_ERR_UNSUPPORTED, "q_dtype must be kv_dtype or RL_DT_F32");
  if (a->batch < 1 || a->q_len < 1 || a->n_q_heads < 1 || a->n_kv_heads < 1 || a->kv_capacity < 1)
    return bad(RL_ERR_INVALID_ARG, "batch, q_len, heads and kv_capacity must be >= 1");
  if (a->head_dim != 64 && a->head_dim != 128) return bad(RL_ERR_UNSUPPORTED, "head_dim must be 64 or 128");
  if (a->n_q_heads % a->n_kv_heads) return bad(RL_ERR_UNSUPPORTED, "n_q_heads must be a multiple of n_kv_heads");
  if (a->kv_capacity > kMaxTokens) return bad(RL_ERR_UNSUPPORTED, "kv_capacity must be at most 2^30");
  if ((long long)a->batch * a->q_len * a->n_q_heads >= (1ll << 31))
    return bad(RL_ERR_UNSUPPORTED, "batch * q_len * n_q_heads must be below 2^31");
  if (!(a->scale >= 0.f) || a->scale > 1e6f) return bad(RL_ERR_INVALID_ARG, "scale must be in [0, 1e6]");
  const int qe = a->q_dtype == RL_DT_F32 ? 4 : 2;
  if (!strides_ok(a->q_stride, 3, qe, 1ll << 59) || !strides_ok(a->out_stride, 3, 2, 1ll << 59))
    return bad(RL_ERR_UNSUPPORTED, "q and out strides must be whole multiples of 16 bytes");
  if (!strides_ok(a->k_stride, 3, 2, 1ll << 39) || !strides_ok(a->v_stride, 3, 2, 1ll << 39))
    return bad(RL_ERR_UNSUPPORTED, "k and v strides must be whole multiples of 16 bytes, below 2^39 elements");
  const int64_t n_out[3] = {a->batch, a->q_len, a->n_q_heads};
  if (!rows_apart(a->out_stride, n_out, a->head_dim)) return bad(RL_ERR_INVALID_ARG, "rows of out overlap");
  memset(o, 0, sizeof(*o));
  o->q_f32 = a->q_dtype == RL_DT_F32;
  o->f16 = a->kv_dtype == RL_DT_F16;
  o->B = a->batch;
  o->Tq = a->q_len;
  o->Hq = a->n_q_heads;
  o->Hkv = a->n_kv_heads;
  o->hd = a->head_dim;
  o->cap = a->kv_capacity;
  o->scale = a->scale > 0.f ? a->scale : 1.f / sqrtf((float)a->head_dim);
  for (int i = 0; i < 3; ++i) {
    o->qs[i] = a->q_stride[i];
    o->os[i] = a->out_stride[i];
    o->kv.ks[i] = a->k_stride[i];
    o->kv.vs[i] = a->v_stride[i];
  }
  o->kv_len_step = 1;
  if (a->kv_capacity > 1 && (a->k_stride[2] == 0 || a->v_stride[2] == 0))
    return bad(RL_ERR_UNSUPPORTED, "k and v token strides must not be 0");
  return RL_OK;
}

}  // namespace

extern "C" rl_status rl_window_attention(const rl_attn_desc* a, const void* d_q, const void* d_k,
                                         const void* d_v, const int32_t* d_kv_len,
                                         const int32_t* d_q_len, int32_t window, int32_t sinks,
                                         void* d_out, float* d_lse, int32_t* d_err, rl_stream_t stream) {
  AttnOpArgs o;
  const rl_status st = check_desc("rl_window_attention", a, &o);
  if (st != RL_OK) return st;
  if (!d_q || !d_k || !d_v || !d_kv_len || !d_out)
    return set_error(RL_ERR_INVALID_ARG, "rl_window_attention: NULL argument");
  if (window < 1 || sinks < 0)
    return set_error(RL_ERR_INVALID_ARG, "rl_window_attention: window must be >= 1 and sinks >= 0");
  if (!aligned16(d_q) || !aligned16(d_k) || !aligned16(d_v) || !aligned16(d_out))
    return set_error(RL_ERR_UNSUPPORTED, "rl_window_attention: q, k, v and out must start on 16-byte boundaries");
  if (d_out == d_q || d_out == d_k || d_out == d_v)
    return set_error(RL_ERR_INVALID_ARG, "rl_window_attention: out overlaps an input");
  o.q = d_q;
  o.out = d_out;
  o.lse = d_lse;
  o.kv.k = d_k;
  o.kv.v = d_v;
  o.kv_len = d_kv_len;
  o.q_len = d_q_len;
  o.window = window < o.cap ? window : o.cap;  // no two positions are further apart
  o.sinks = sinks < o.cap ? sinks : o.cap;
  o.err = d_err;
  const cudaError_t e = launch_window_attention(o, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return set_error(RL_ERR_CUDA, cudaGetErrorString(e));
  return RL_OK;
}

extern "C" rl_status rl_shared_prefix_workspace(const rl_attn_desc* a, int32_t prefix_len, uint64_t* bytes) {
  AttnOpArgs o;
  const rl_status st = check_desc("rl_shared_prefix_workspace", a, &o);
  if (st != RL_OK) return st;
  if (!bytes || prefix_len < 0)
    return set_error(RL_ERR_INVALID_ARG, "rl_shared_prefix_workspace: bytes is NULL or prefix_len below 0");
  if (prefix_len > kMaxTokens)
    return set_error(RL_ERR_UNSUPPORTED, "rl_shared_prefix_workspace: prefix_len must be at most 2^30");
  *bytes = shared_prefix_ws_bytes(o.B, o.Hq, o.Hkv, o.hd, prefix_len);
  return RL_OK;
}

extern "C" rl_status rl_shared_prefix_attention(const rl_attn_desc* a, const void* d_q,
                                                const void* d_k_prefix, const void* d_v_prefix,
                                                int32_t prefix_len, const int64_t prefix_stride[4],
                                                const void* d_k, const void* d_v,
                                                const int32_t* d_kv_len, void* d_out, float* d_lse,
                                                void* d_ws, uint64_t ws_bytes, int32_t* d_err,
                                                rl_stream_t stream) {
  AttnOpArgs o;
  const rl_status st = check_desc("rl_shared_prefix_attention", a, &o);
  if (st != RL_OK) return st;
  if (o.Tq != 1) return set_error(RL_ERR_UNSUPPORTED, "rl_shared_prefix_attention: q_len must be 1");
  if (!d_q || !d_k || !d_v || !d_kv_len || !d_out || !d_ws)
    return set_error(RL_ERR_INVALID_ARG, "rl_shared_prefix_attention: NULL argument");
  if (prefix_len < 0 || (prefix_len > 0 && (!d_k_prefix || !d_v_prefix || !prefix_stride)))
    return set_error(RL_ERR_INVALID_ARG, "rl_shared_prefix_attention: prefix_len below 0, or a prefix argument NULL");
  if (prefix_len > kMaxTokens)
    return set_error(RL_ERR_UNSUPPORTED, "rl_shared_prefix_attention: prefix_len must be at most 2^30");
  if (!aligned16(d_q) || !aligned16(d_k) || !aligned16(d_v) || !aligned16(d_out) || !aligned16(d_ws))
    return set_error(RL_ERR_UNSUPPORTED,
                     "rl_shared_prefix_attention: q, k, v, out and the workspace must start on 16-byte boundaries");
  if (d_out == d_q || d_out == d_k || d_out == d_v)
    return set_error(RL_ERR_INVALID_ARG, "rl_shared_prefix_attention: out overlaps an input");
  if (ws_bytes < shared_prefix_ws_bytes(o.B, o.Hq, o.Hkv, o.hd, prefix_len))
    return set_error(RL_ERR_INVALID_ARG, "rl_shared_prefix_attention: workspace too small");
  if (prefix_len > 0) {
    if (!aligned16(d_k_prefix) || !aligned16(d_v_prefix) || !strides_ok(prefix_stride, 4, 2, 1ll << 39))
      return set_error(RL_ERR_UNSUPPORTED,
                       "rl_shared_prefix_attention: the prefix must start on 16-byte boundaries, strides whole "
                       "multiples of 16 bytes below 2^39 elements");
    if (prefix_len > 1 && (prefix_stride[1] == 0 || prefix_stride[3] == 0))
      return set_error(RL_ERR_UNSUPPORTED, "rl_shared_prefix_attention: the prefix's token strides must not be 0");
    o.pre.k = d_k_prefix;
    o.pre.v = d_v_prefix;
    o.pre.ks[1] = prefix_stride[0];
    o.pre.ks[2] = prefix_stride[1];
    o.pre.vs[1] = prefix_stride[2];
    o.pre.vs[2] = prefix_stride[3];
    o.P = prefix_len;
  }
  o.q = d_q;
  o.out = d_out;
  o.lse = d_lse;
  o.kv.k = d_k;
  o.kv.v = d_v;
  o.kv_len = d_kv_len;
  o.window = o.cap;
  o.err = d_err;
  o.ws = d_ws;
  const cudaError_t e = launch_shared_prefix_attention(o, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return set_error(RL_ERR_CUDA, cudaGetErrorString(e));
  return RL_OK;
}
