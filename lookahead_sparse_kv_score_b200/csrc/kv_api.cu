// The C ABI of the 8-bit KV cache and of the rotary positions: argument checks, workspace
// layout and dispatch.  Every entry point is declared and documented in include/lsa.h.
#include <algorithm>
#include <cmath>

#include "kv_common.cuh"

namespace lsa {
namespace {

int log2_exact(int x) {   // -1 unless x is a power of two
  if (x <= 0 || (x & (x - 1)) != 0) return -1;
  int k = 0;
  while ((1 << k) < x) ++k;
  return k;
}

// Fills g from the arguments common to the cache's calls; LSA_OK or an error of `who`.
int make_geom(const char* who, int B, int N, int G, int W, int block, int page, int seq_pages, int pages,
              const int32_t* table, const void* rows, const float* scale, KvGeom& g) {
  if (B < 0 || N < 0 || G < 1 || W < 16) return fail(LSA_ERR_INVALID_ARG, "%s: bad size (B %d, N %d, G %d, W %d)", who, B, N, G, W);
  if (W % 16 != 0) return fail(LSA_ERR_INVALID_ARG, "%s: W = %d is not a multiple of 16", who, W);
  g.block_log = log2_exact(block);
  g.page_log = log2_exact(page);
  if (g.block_log < 0 || block > 128) return fail(LSA_ERR_INVALID_ARG, "%s: block = %d (a power of two up to 128)", who, block);
  if (g.page_log < 0) return fail(LSA_ERR_INVALID_ARG, "%s: page = %d (a power of two)", who, page);
  if (seq_pages < 0 || pages < 0) return fail(LSA_ERR_INVALID_ARG, "%s: negative page count", who);
  const long long rows_all = static_cast<long long>(pages) * page * G;
  if (rows_all > 0x7fffffffll) return fail(LSA_ERR_UNSUPPORTED, "%s: %lld rows (at most 2^31 - 1)", who, rows_all);
  g.B = B; g.N = N; g.G = G; g.W = W;
  g.seq_pages = seq_pages;
  g.pages = pages;
  g.n_blocks = static_cast<int>((static_cast<long long>(N) + block - 1) / block);
  g.n_pages = static_cast<int>((static_cast<long long>(N) + page - 1) / page);
  if (B == 0 || N == 0) return LSA_OK;
  if (!rows || !scale) return fail(LSA_ERR_INVALID_ARG, "%s: rows or scale is null", who);
  if (!aligned(rows, 16) || !aligned(scale, 4) || (table && !aligned(table, 4)))
    return fail(LSA_ERR_INVALID_ARG, "%s: misaligned pointer (rows 16 bytes, scale and table 4)", who);
  if (!table && static_cast<long long>(seq_pages) * (B - 1) + g.n_pages > pages)
    return fail(LSA_ERR_INVALID_ARG, "%s: %d pages cannot hold %d sequences of %d pages", who, pages, B, g.n_pages);
  if (!table && seq_pages > 0 && seq_pages < g.n_pages)
    return fail(LSA_ERR_INVALID_ARG, "%s: seq_pages = %d, a sequence has %d", who, seq_pages, g.n_pages);
  g.table = table;
  g.rows = static_cast<uint8_t*>(const_cast<void*>(rows));
  g.scale = const_cast<float*>(scale);
  return LSA_OK;
}

struct AttendWs {
  int cols;          // query columns of a block on the tensor cores, 0: CUDA cores
  int cluster, team, splits;
  size_t o, m, l, total;
};

AttendWs attend_ws(int B, int Tq, int N, int H, int G, int d, int dv, int voff, int qdt, int sinks, int window, int cap) {
  AttendWs w{};
  const int ncol = Tq * (H / G);
  long long most = window < 0 ? N : std::min<long long>(N, static_cast<long long>(sinks) + window + Tq - 1);
  most += cap + (window > 0 ? 64 : 0);         // and the numbering's empty places around a window
  const int b1 = std::max(B, 1), n1 = std::max(ncol, 1);
  w.cols = N <= (1 << 30) ? kv_attend_columns_tc(b1, G, n1, most, d, dv, voff, qdt) : 0;   // token words have 30 bits
  w.cluster = 1;
  if (w.cols > 0) kv_attend_parts_tc(b1, G, n1, w.cols, d, dv, voff, most, w.cluster, w.splits);
  else kv_attend_parts_simt(b1, G, n1, most, w.team, w.splits);
  const size_t cols = static_cast<size_t>(B) * G * w.splits * ncol;
  size_t off = 0;
  auto take = [&](size_t bytes) { const size_t at = off; off = align_up(off + bytes, 256); return at; };
  if (w.splits > 1) {
    w.o = take(cols * dv * 4);
    w.m = take(cols * 4);
    w.l = take(cols * 4);
  }
  w.total = std::max<size_t>(off, 256);
  return w;
}

int attend_shape(int B, int Tq, int N, int H, int G, int d, int dv, int voff, int W, int qdt, int sinks, int cap) {
  if (B < 0 || Tq < 0 || N < 0 || H < 1 || G < 1 || d < 1 || dv < 1 || voff < 0 || sinks < 0 || cap < 0)
    return fail(LSA_ERR_INVALID_ARG, "kv_attend: bad size");
  if (H % G != 0) return fail(LSA_ERR_INVALID_ARG, "kv_attend: %d heads do not divide into %d KV heads", H, G);
  if (d > W || static_cast<long long>(voff) + dv > W)
    return fail(LSA_ERR_INVALID_ARG, "kv_attend: columns [0, %d) and [%d, %d) of a row of %d", d, voff, voff + dv, W);
  if (qdt != LSA_F32 && qdt != LSA_BF16) return fail(LSA_ERR_UNSUPPORTED, "kv_attend: query dtype %d", qdt);
  if (d > 576 || dv > 512 || voff + dv > 1024)
    return fail(LSA_ERR_UNSUPPORTED, "kv_attend: d = %d (at most 576), dv = %d (at most 512), voff + dv = %d (at most 1024)", d, dv, voff + dv);
  if (static_cast<long long>(N) + cap > 0x7fff0000ll)
    return fail(LSA_ERR_UNSUPPORTED, "kv_attend: N + cap = %lld (at most 2^31 - 2^16)", static_cast<long long>(N) + cap);
  if (static_cast<long long>(Tq) * (H / G) > 65536)
    return fail(LSA_ERR_UNSUPPORTED, "kv_attend: %lld query columns of a KV head (at most 65536)", static_cast<long long>(Tq) * (H / G));
  if (static_cast<long long>(B) * Tq * H > (1ll << 24))
    return fail(LSA_ERR_UNSUPPORTED, "kv_attend: B * Tq * H = %lld (at most 2^24)", static_cast<long long>(B) * Tq * H);
  return LSA_OK;
}

}  // namespace
}  // namespace lsa

using namespace lsa;

extern "C" {

int lsa_kv_write(int B, int T, int N, int G, int W, int xdt, const void* x, size_t x_stride, const int32_t* start,
                 const int32_t* count, int block, int page, int seq_pages, int pages, const int32_t* table,
                 void* rows, float* scale, int32_t* status, void* stream) {
  const CallRange range("lsa_kv_write");
  clear_error();
  KvGeom g{};
  const int rc = make_geom("kv_write", B, N, G, W, block, page, seq_pages, pages, table, rows, scale, g);
  if (rc != LSA_OK) return rc;
  if (T < 0) return fail(LSA_ERR_INVALID_ARG, "kv_write: T = %d", T);
  if (xdt != LSA_F32 && xdt != LSA_BF16) return fail(LSA_ERR_UNSUPPORTED, "kv_write: dtype %d", xdt);
  if (B == 0 || T == 0 || N == 0) return LSA_OK;
  if (!x || !start) return fail(LSA_ERR_INVALID_ARG, "kv_write: x or start is null");
  const size_t es = xdt == LSA_F32 ? 4 : 2;
  if (!aligned(x, 16) || x_stride * es % 16 != 0 || !aligned(start, 4) || (count && !aligned(count, 4)))
    return fail(LSA_ERR_INVALID_ARG, "kv_write: misaligned pointer or stride (x and its rows 16 bytes)");
  if (x_stride < static_cast<size_t>(G) * W)
    return fail(LSA_ERR_INVALID_ARG, "kv_write: x_stride = %zu is shorter than a token's %zu elements", x_stride, static_cast<size_t>(G) * W);
  if (B > 1 && !table && seq_pages == 0)
    return fail(LSA_ERR_INVALID_ARG, "kv_write: %d sequences would write the same rows (no table and seq_pages = 0)", B);
  if (static_cast<long long>(B) * T * G > 0x3fffffffll)
    return fail(LSA_ERR_UNSUPPORTED, "kv_write: B * T * G = %lld (at most 2^30 - 1)", static_cast<long long>(B) * T * G);
  return launch_kv_write(g, T, xdt, x, x_stride, start, count, status, static_cast<cudaStream_t>(stream));
}

int lsa_kv_read(int B, int N, int G, int W, const int32_t* idx, int cap, const int32_t* count, int block, int page,
                int seq_pages, int pages, const int32_t* table, const void* rows, const float* scale, int odt,
                void* out, int32_t* status, void* stream) {
  const CallRange range("lsa_kv_read");
  clear_error();
  KvGeom g{};
  const int rc = make_geom("kv_read", B, N, G, W, block, page, seq_pages, pages, table, rows, scale, g);
  if (rc != LSA_OK) return rc;
  if (cap < 0) return fail(LSA_ERR_INVALID_ARG, "kv_read: cap = %d", cap);
  if (odt != LSA_F32 && odt != LSA_BF16) return fail(LSA_ERR_UNSUPPORTED, "kv_read: dtype %d", odt);
  if (B == 0 || cap == 0 || N == 0) return LSA_OK;
  if (!out) return fail(LSA_ERR_INVALID_ARG, "kv_read: out is null");
  if (!aligned(out, 16) || (idx && !aligned(idx, 4)) || (count && !aligned(count, 4)))
    return fail(LSA_ERR_INVALID_ARG, "kv_read: misaligned pointer (out 16 bytes)");
  if (!idx && cap > N) return fail(LSA_ERR_INVALID_ARG, "kv_read: cap = %d tokens of %d without a list", cap, N);
  return launch_kv_read(g, idx, cap, count, odt, out, status, static_cast<cudaStream_t>(stream));
}

size_t lsa_kv_attend_workspace_bytes(int B, int Tq, int N, int H, int G, int d, int dv, int voff, int W, int qdt,
                                     int sinks, int window, int cap) {
  if (attend_shape(B, Tq, N, H, G, d, dv, voff, W, qdt, sinks, cap) != LSA_OK) return 0;
  return attend_ws(B, Tq, N, H, G, d, dv, voff, qdt, sinks, window, cap).total;
}

int lsa_kv_attend(int B, int Tq, int N, int H, int G, int d, int dv, int voff, int W, int qdt, const void* q,
                  float sm_scale, const int32_t* length, int sinks, int window, const int32_t* idx, int cap,
                  const int32_t* count, int block, int page, int seq_pages, int pages, const int32_t* table,
                  const void* rows, const float* scale, void* out, float* lse, int32_t* status, void* workspace,
                  size_t workspace_bytes, void* stream) {
  const CallRange range("lsa_kv_attend");
  clear_error();
  KvGeom g{};
  int rc = make_geom("kv_attend", B, N, G, W, block, page, seq_pages, pages, table, rows, scale, g);
  if (rc != LSA_OK) return rc;
  if (!idx || N == 0) {   // no list, or none of its entries can be a token
    idx = nullptr;
    cap = 0;
  }
  rc = attend_shape(B, Tq, N, H, G, d, dv, voff, W, qdt, sinks, cap);
  if (rc != LSA_OK) return rc;
  if (!(std::fabs(sm_scale) <= 3.4e38f)) return fail(LSA_ERR_INVALID_ARG, "kv_attend: sm_scale is not finite");
  if (B == 0 || Tq == 0) return LSA_OK;
  if (!q || !length || !out || (idx && !count)) return fail(LSA_ERR_INVALID_ARG, "kv_attend: null pointer (a list needs its counts)");
  if (!aligned(q, 16) || !aligned(out, 16) || (lse && !aligned(lse, 4)) || !aligned(length, 4) ||
      (idx && (!aligned(idx, 4) || !aligned(count, 4))))
    return fail(LSA_ERR_INVALID_ARG, "kv_attend: misaligned pointer");
  const AttendWs ws = attend_ws(B, Tq, N, H, G, d, dv, voff, qdt, sinks, window, cap);
  if (!workspace || workspace_bytes < ws.total || !aligned(workspace, 256))
    return fail(LSA_ERR_NOMEM, "kv_attend: workspace %zu bytes (need %zu, 256-byte aligned)", workspace_bytes, ws.total);
  KvAttendArgs a{};
  a.g = g;
  a.Tq = Tq; a.H = H; a.d = d; a.dv = dv; a.voff = voff; a.qdt = qdt;
  a.sm = sm_scale;
  a.sinks = sinks; a.window = window; a.cap = cap;
  a.q = q; a.length = length; a.idx = idx; a.count = count;
  a.out = out; a.lse = lse; a.status = status;
  a.splits = ws.splits;
  uint8_t* base = static_cast<uint8_t*>(workspace);
  a.part_o = reinterpret_cast<float*>(base + ws.o);
  a.part_m = reinterpret_cast<float*>(base + ws.m);
  a.part_l = reinterpret_cast<float*>(base + ws.l);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  rc = ws.cols > 0 ? launch_kv_attend_tc(a, ws.cols, ws.cluster, st) : launch_kv_attend_simt(a, ws.team, st);
  if (rc != LSA_OK || a.splits == 1) return rc;
  return launch_kv_attend_combine(a, st);
}

int lsa_rope(int R, int H, int rot, int half, int dt, const void* x, long long x_token, long long x_head,
             const int32_t* pos, const double* freq, float mscale, int inverse, void* out, long long o_token,
             long long o_head, void* stream) {
  const CallRange range("lsa_rope");
  clear_error();
  if (R < 0 || H < 0 || rot < 0 || rot % 2 != 0 || rot > 1024)
    return fail(LSA_ERR_INVALID_ARG, "rope: R %d, H %d, rot %d (even, at most 1024)", R, H, rot);
  if (dt != LSA_F32 && dt != LSA_BF16) return fail(LSA_ERR_UNSUPPORTED, "rope: dtype %d", dt);
  if (R == 0 || H == 0 || rot == 0) return LSA_OK;
  if (static_cast<long long>(H) * rot > (1ll << 24)) return fail(LSA_ERR_UNSUPPORTED, "rope: H * rot = %lld (at most 2^24)", static_cast<long long>(H) * rot);
  if (!x || !pos || !freq || !out) return fail(LSA_ERR_INVALID_ARG, "rope: null pointer");
  const size_t es = dt == LSA_F32 ? 4 : 2;
  if (!aligned(x, es) || !aligned(out, es) || !aligned(pos, 4) || !aligned(freq, 8))
    return fail(LSA_ERR_INVALID_ARG, "rope: misaligned pointer");
  if ((H > 1 && (x_head < rot || o_head < rot)) || (R > 1 && (x_token < rot || o_token < rot)))
    return fail(LSA_ERR_INVALID_ARG, "rope: a stride shorter than the rotated part");
  // The output's tokens and heads must not share elements: the larger stride spans the smaller.
  const long long s1 = std::min(o_token, o_head), s2 = std::max(o_token, o_head), n1 = o_token < o_head ? R : H;
  if (R > 1 && H > 1 && s2 < (n1 - 1) * s1 + rot)
    return fail(LSA_ERR_INVALID_ARG, "rope: output strides %lld and %lld overlap", o_token, o_head);
  RopeArgs a{};
  a.R = R; a.H = H; a.rot = rot; a.half = half != 0; a.dt = dt; a.inverse = inverse != 0;
  a.x = x; a.x_token = x_token; a.x_head = x_head;
  a.pos = pos; a.freq = freq; a.mscale = mscale;
  a.out = out; a.o_token = o_token; a.o_head = o_head;
  return launch_rope(a, static_cast<cudaStream_t>(stream));
}

int lsa_rope_frequencies(int rot, double base, double factor, double original, double fast, double slow, double* freq) {
  clear_error();
  if (rot < 0 || rot % 2 != 0 || rot > 1024) return fail(LSA_ERR_INVALID_ARG, "rope_frequencies: rot %d (even, at most 1024)", rot);
  if (rot > 0 && !freq) return fail(LSA_ERR_INVALID_ARG, "rope_frequencies: freq is null");
  if (!(base > 1.0) || !(factor >= 1.0) || !std::isfinite(base) || !std::isfinite(factor))
    return fail(LSA_ERR_INVALID_ARG, "rope_frequencies: base %g (above 1), factor %g (1 or more)", base, factor);
  if (factor > 1.0 && (!(original > 0.0) || !(fast > slow) || !(slow > 0.0) || !std::isfinite(original) || !std::isfinite(fast)))
    return fail(LSA_ERR_INVALID_ARG, "rope_frequencies: original %g, fast %g, slow %g", original, fast, slow);
  double lo = 0.0, hi = 0.0;
  if (factor > 1.0) {
    const double two_pi = 6.283185307179586476925286766559;
    auto at = [&](double turns) { return rot * std::log(original / (turns * two_pi)) / (2.0 * std::log(base)); };
    lo = std::max(std::floor(at(fast)), 0.0);
    hi = std::min(std::ceil(at(slow)), rot - 1.0);   // may lie past the last pair, rot / 2 - 1
  }
  for (int i = 0; i < rot / 2; ++i) {
    double f = std::pow(base, -2.0 * i / rot);
    if (factor > 1.0) {
      const double ramp = std::min(std::max((i - lo) / std::max(hi - lo, 1e-3), 0.0), 1.0);
      f = f * (1.0 - ramp) + f / factor * ramp;
    }
    freq[i] = f;
  }
  return LSA_OK;
}

}  // extern "C"
