// Geometry of the 8-bit KV cache and the set of tokens an attention call sees, shared by the
// cache's write, read and attention kernels.
#pragma once

#include "lsa_common.cuh"

namespace lsa {

// Rows [pages][page][G][W] of e4m3 codes; scale [B][ceil(N/block)][G]; table [B][ceil(N/page)]
// or null.  page and block are powers of two.
struct KvGeom {
  int B, N, G, W;
  int block_log, page_log;
  int seq_pages, pages;
  int n_blocks, n_pages;    // per sequence: ceil(N / block), ceil(N / page)
  const int32_t* table;
  uint8_t* rows;
  float* scale;
};

// Page of token t (0 <= t < N) of sequence b as the table has it.
__device__ __forceinline__ int kv_page(const KvGeom& g, int b, int t) {
  const int p = t >> g.page_log;
  return g.table != nullptr ? g.table[static_cast<size_t>(b) * g.n_pages + p] : p;
}

// Row of a token on page p, in units of G * W bytes, or -1 where the table has no page for it or
// the page lies outside the pool.
__device__ __forceinline__ long long kv_row_of(const KvGeom& g, int b, int t, int p) {
  if (p < 0 || (g.seq_pages > 0 && p >= g.seq_pages)) return -1;
  const long long phys = static_cast<long long>(b) * g.seq_pages + p;
  if (phys >= g.pages) return -1;
  return (phys << g.page_log) + (t & ((1 << g.page_log) - 1));
}
__device__ __forceinline__ long long kv_row(const KvGeom& g, int b, int t) { return kv_row_of(g, b, t, kv_page(g, b, t)); }

__device__ __forceinline__ size_t kv_scale_at(const KvGeom& g, int b, int t, int head) {
  return (static_cast<size_t>(b) * g.n_blocks + (t >> g.block_log)) * g.G + head;
}

// ------------------------------------------------------------------ attention
struct KvAttendArgs {
  KvGeom g;
  int Tq, H, d, dv, voff, qdt;
  float sm;                   // softmax scale
  int sinks, window, cap;
  const void* q;              // [B][Tq][H][d]
  const int32_t* length;      // [B]
  const int32_t* idx;         // [B][cap] or null
  const int32_t* count;       // [B]
  void* out;                  // [B][Tq][H][dv]
  float* lse;                 // [B][Tq][H] or null
  int32_t* status;
  int splits;                 // parts a sequence's tokens are divided into
  float* part_o;              // workspace [B*G][splits][ncol][dv], splits > 1
  float* part_m;              // workspace [B*G][splits][ncol]: reference exponent (base 2)
  float* part_l;              // workspace [B*G][splits][ncol]: sum of 2^(x - m)
};

// The tokens one sequence's queries can see, in one numbering v = 0 .. total-1: the first
// tokens, the window (of all queries together) and the listed entries.  The window starts on a
// multiple of 16 tokens, and the first tokens are padded to 32 places, so that runs of a
// page's rows stay runs of places; the places without a token are empty.
struct KvSpan {
  int len, first, pad, lo, start, n_main, total;
};

__device__ __forceinline__ KvSpan kv_span(const KvAttendArgs& a, int b) {
  KvSpan s;
  s.len = min(max(a.length[b], 0), a.g.N);
  const int listed = a.idx != nullptr ? max(0, min(a.count[b], a.cap)) : 0;
  s.first = s.pad = s.lo = s.start = 0;
  s.n_main = s.len;
  if (a.window >= 0) {
    s.first = min(a.sinks, s.len);
    // lowest position in any query's window; len - Tq is the first query's position
    const long long lo = static_cast<long long>(s.len) - a.Tq - a.window + 1;
    s.lo = static_cast<int>(lo > s.first ? lo : s.first);
    s.start = max(s.first, s.lo & ~15);
    const bool window = a.window > 0 && s.len > s.lo;
    s.pad = window && s.first > 0 && s.first <= 0x7fffffff - 31 ? (s.first + 31) & ~31 : s.first;
    s.n_main = s.pad + (window ? s.len - s.start : 0);
  }
  s.total = s.n_main + listed;
  return s;
}

// Whether the query at position p sees token t of the first tokens or of the window.
__device__ __forceinline__ bool kv_sees(const KvAttendArgs& a, int t, int p) {
  return t <= p && (a.window < 0 || t < a.sinks || t > p - static_cast<long long>(a.window));
}

// Token v of the numbering, or -1 for an empty place and for a list entry that is padding or
// out of range.
__device__ __forceinline__ int kv_token(const KvAttendArgs& a, const KvSpan& s, int b, int v, bool& main) {
  main = v < s.n_main;
  if (main) {
    if (v < s.pad) return v < s.first ? v : -1;
    const int t = s.start + (v - s.pad);
    return t < s.lo ? -1 : t;
  }
  const int e = a.idx[static_cast<size_t>(b) * a.cap + (v - s.n_main)];
  if (e >= s.len) {
    raise_status(a.status, LSA_ERR_RANGE);
    return -1;
  }
  return e < 0 ? -1 : e;
}

// ln(2^m sum).  The exponents are added first: with scales far from 1 they are large and cancel, and a
// rounded log2 of the whole sum would cost what the difference has.
__device__ __forceinline__ float kv_lse(float m, float sum) {
  if (sum == 0.f) return -INFINITY;
  int e;
  const float f = frexpf(sum, &e);
  return ((m + static_cast<float>(e)) + log2f(f)) * 0.693147180559945f;
}

// The tensor-core path: query columns of a block (16, 32 or 64; 0: shape not supported), blocks
// of a cluster and clusters of a unit (KvAttendArgs::splits).
int kv_attend_columns_tc(int B, int G, int ncol, long long max_tokens, int d, int dv, int voff, int qdt);
void kv_attend_parts_tc(int B, int G, int ncol, int C, int d, int dv, int voff, long long max_tokens, int& cluster, int& groups);
int launch_kv_attend_tc(const KvAttendArgs& a, int C, int cluster, cudaStream_t s);
// The CUDA-core path: warps of a column, and parts of a unit's tokens (KvAttendArgs::splits).
void kv_attend_parts_simt(int B, int G, int ncol, long long max_tokens, int& team, int& splits);
int launch_kv_attend_simt(const KvAttendArgs& a, int team, cudaStream_t s);
int launch_kv_attend_combine(const KvAttendArgs& a, cudaStream_t s);

// ------------------------------------------------------------------ cache and rotation
int launch_kv_write(const KvGeom& g, int T, int xdt, const void* x, size_t x_stride, const int32_t* start,
                    const int32_t* count, int32_t* status, cudaStream_t s);
int launch_kv_read(const KvGeom& g, const int32_t* idx, int cap, const int32_t* count, int odt, void* out,
                   int32_t* status, cudaStream_t s);

struct RopeArgs {
  int R, H, rot, half, dt, inverse;
  const void* x;
  long long x_token, x_head;
  const int32_t* pos;
  const double* freq;
  float mscale;
  void* out;
  long long o_token, o_head;
};
int launch_rope(const RopeArgs& a, cudaStream_t s);

}  // namespace lsa
