// What the operators over packed rows and over the 4-bit paged cache share:
// arguments, the sequence of a row, lengths, pages.
#pragma once

#include "attn_ops.cuh"

namespace river {

struct PackedArgs {
  int f16, B, N, max_rows, Hq, Hkv, hd;
  float scale;                           // natural-log units
  long long qs[2], ks[2], vs[2], os[2];  // row, head
  const void *q, *k, *v;
  void* out;
  float* lse;
  const int *start, *kv_len;             // start: null, one row each
  int* err;
};
struct Kv4Args {
  int n_pages, page_log;                 // token rows of a page: 1 << page_log
  unsigned char *kc, *vc;                // codes
  uint32_t *km, *vm;                     // (step, minimum) pairs
  long long kc_step, vc_step, km_step, vm_step;  // from page to page: bytes, pairs
  const int* table;
  long long table_step;
  int width;
};

// The checks of a packed call (kv4_rows.cu); fills `o`.
enum { kUsesQ = 1, kUsesK = 2, kUsesV = 4, kUsesOut = 8 };
rl_status check_packed(const char* who, const rl_packed_desc* p, int reads, int writes, PackedArgs* o);
rl_status check_kv4(const char* who, const rl_kv4* c, const PackedArgs& p, Kv4Args* o);
bool op_aligned16(const void* p);
rl_status op_error(const char* who, rl_status st, const char* what);

namespace attn {

// Rows of sequence b: `all` from `first` on, of which n <= max_rows count.
struct Span {
  int first, n, all;
};
__device__ __forceinline__ Span seq_span(const PackedArgs& a, int b, bool report) {
  if (!a.start) return Span{b, b < a.N, 1};
  const int s0 = __ldg(a.start + b), s1 = __ldg(a.start + b + 1);
  const int f = max(0, min(s0, a.N)), e = max(f, min(s1, a.N));
  if (report && a.err && e - f > a.max_rows) atomicOr(a.err, RL_DEVERR_CAPACITY);
  return Span{f, min(e - f, a.max_rows), e - f};
}

// The sequence that packed row r belongs to, by a search 32 ways at a time;
// -1: none.  The same for a warp's lanes.
__device__ __forceinline__ int seq_of_row(const PackedArgs& a, int r, int lane) {
  if (!a.start) return r < a.B ? r : -1;
  int lo = 0, hi = a.B;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) >> 5, i = lo + lane * step;
    const unsigned le = __ballot_sync(0xffffffffu, lane == 0 || (i < hi && __ldg(a.start + i) <= r));
    lo += (31 - __clz(le)) * step;
    hi = min(hi, lo + step);
  }
  return __ldg(a.start + lo) <= r && r < __ldg(a.start + lo + 1) ? lo : -1;
}

// Every entry of start in its place (the first block's threads look).
__device__ __forceinline__ void check_start(const PackedArgs& a) {
  if (!a.start || !a.err || blockIdx.x != 0) return;
  for (int b = threadIdx.x; b <= a.B; b += blockDim.x) {
    const int s = __ldg(a.start + b);
    if (s < 0 || s > a.N || (b > 0 && s < __ldg(a.start + b - 1))) atomicOr(a.err, RL_DEVERR_CAPACITY);
  }
}

// Page i of sequence b; -1 (reported) outside the cache.
__device__ __forceinline__ int page_at(const PackedArgs& a, const Kv4Args& c, int b, int i) {
  const int p = __ldg(c.table + (long long)b * c.table_step + i);
  if ((unsigned)p < (unsigned)c.n_pages) return p;
  if (a.err) atomicOr(a.err, RL_DEVERR_CAPACITY);
  return -1;
}
// Row `row` of head hk in a page: its number among the page's rows.
__device__ __forceinline__ long long page_row(const Kv4Args& c, int hk, int row) {
  return ((long long)hk << c.page_log) + row;
}

}  // namespace attn

cudaError_t launch_kv4_append(const PackedArgs& p, const Kv4Args& c, const float2* rope, int rope_len, cudaStream_t s);
cudaError_t launch_kv4_read(const PackedArgs& p, const Kv4Args& c, void* k, void* v, cudaStream_t s);
size_t kv4_attention_ws_bytes(const PackedArgs& p);
bool kv4_attention_fits(const PackedArgs& p, const Kv4Args& c);
cudaError_t launch_kv4_attention(const PackedArgs& p, const Kv4Args& c, void* ws, cudaStream_t s);
cudaError_t launch_packed_attention(const PackedArgs& p, cudaStream_t s);

}  // namespace river
