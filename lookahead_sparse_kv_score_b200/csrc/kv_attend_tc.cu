// Attention over the 8-bit KV cache on the tensor cores of sm_100a: TMA row gathers ->
// shared memory -> tcgen05.mma -> tensor memory, one pass with a running reference exponent.
//
// The cached codes are the MMA's operands as they lie in memory: nothing is decoded to 16
// bits, so a tile crosses shared memory once and both products read the same bytes.  A
// tile is 128 tokens of one KV head; the query columns c (query token and head of its group)
// of a unit are the MMA's N, at most 64 (C) a block:
//     S^T [128 tokens][2C] = K [128][d] . [hi | lo]^T,       q = s_c (hi + lo), both e4m3
//     O^T [128 columns of V][C] += V^T [128][128 tokens] . (P_hi + P_lo) [128 tokens][C].
// With tokens as M in the first product and value columns as M in the second, a few query
// columns cost a few columns of N instead of a padded M.
//
// Rounding.  A bf16 query element has 8 significant bits; scaled by a power of two to at most
// 448, an e4m3 term holds the first four and a second one the rest, exactly, except
// below 2^-10 / 224 of the row's largest element.  A weight P'' (see below) is held as an e4m3
// and an e5m2 term: half a step of each is 2^-4 * 2^-3 = 2^-7 of the weight at most (rms
// 1.2e-3, below the bf16 rounding of the result), and the e5m2 range keeps weights down to
// 2^-17, 2^-23 of the reference weight; with at most 16384 tokens in a part the weights lost
// below that are less than 2^-9 of the sum.  Scores, the sum of the weights and the
// accumulators are fp32.
//
// Scales.  y_tc = sm log2(e) scale_t (q_c . k_t) + log2(scale_t); the value weight is
// P''_tc = 2^(y_tc - r_c) and the softmax weight P''_tc / scale_t, so one exponential serves
// both sums and the scale never multiplies the codes.  r_c is set so that the largest weight
// seen is 64 and kept until a weight would pass 448: then the block's O^T columns are
// multiplied by 2^(r_old - r_new) in tensor memory.  That is rare after the first tile, so the
// cross-lane maxima are only computed then; otherwise a tile costs one vote.
//
// Roles (12 warps): warp 0 gathers rows (lane l the tile's tokens 4l .. 4l+3, four rows a TMA
// instruction and 128-byte chunk) and writes the tokens' scales; warp 1 issues the MMAs,
// S of the next tile before O of this one; warps 4-11 hold one token a lane and half of the
// columns each.  Waits are bounded; on expiry LSA_ERR_TIMEOUT is raised, MMAs and copies in
// flight are drained and the tensor memory is freed.
#include <cuda.h>

#include <algorithm>
#include <climits>

#include "kv_common.cuh"
#include "tc_ptx.cuh"

namespace lsa {
namespace {

using namespace tc;

constexpr int kTile = 128;
constexpr int kThreads = 384;
constexpr int kSmemLimit = 227 * 1024;
constexpr int kChunkBytes = kTile * 128;      // 128 columns of a tile, 128-byte swizzle
constexpr int kTailBytes = kTile * 64;        // the last 64 key columns, 64-byte swizzle
constexpr int kMaxStages = 6;
constexpr int kBars = 40;                     // 8-byte words of barriers and flags
constexpr float kUnset = -3.0e38f;            // reference exponent before any token was seen
constexpr float kTarget = 6.f;                // the largest weight is set to 2^6
constexpr float kLimit = 8.8f;                // 2^8.8 < 448: reference kept up to here
constexpr int kListFlag = 1 << 30;            // token word: a list entry
constexpr int kAllFlag = INT_MIN;             // token word: every query of the unit sees it

// Which 128-column chunks of a row a tile holds, and the shared-memory plan.
struct Plan {
  int n_k;          // key chunks, the tail among them
  int tail;         // 1 when the last key chunk is a 64-column tail
  int v0, n_v;      // value chunks
  int n_full;       // 128-column chunks in a stage
  int ksteps;       // 32-element steps of the first product
  int stages, tstages;
  int q_bytes, p_off, q_off, t_off, i_off, m_off, smem;
};

__host__ __device__ inline int plan_v_slot(const Plan& p, int chunk) {   // ring slot of a value chunk
  const int n_kf = p.n_k - p.tail;
  if (chunk < n_kf) return chunk;
  return n_kf + chunk - (p.v0 > n_kf ? p.v0 : n_kf);
}

Plan make_plan(int d, int dv, int voff, int C) {
  Plan p{};
  p.n_k = (d + 127) / 128;
  p.v0 = voff / 128;
  const int v1 = (voff + dv + 127) / 128;
  p.n_v = v1 - p.v0;
  const int rest = d - (p.n_k - 1) * 128;
  p.tail = rest <= 64 && !(p.n_k - 1 >= p.v0 && p.n_k - 1 < v1) ? 1 : 0;
  const int n_kf = p.n_k - p.tail;
  p.n_full = n_kf + std::max(0, v1 - std::max(p.v0, n_kf));
  p.ksteps = (d + 31) / 32;
  p.q_bytes = 2 * C * (n_kf * 128 + p.tail * 64);
  const int stage = p.n_full * kChunkBytes;
  const int fixed = p.q_bytes + kChunkBytes /* weights */ + kBars * 8 + 8 * C + 2 * C;
  // whole stages with their tails while they fit, then whole stages on one tail
  const int per = stage + p.tail * kTailBytes + kTile * 8 + 8;
  p.stages = std::min(kMaxStages, (kSmemLimit - fixed) / per);
  p.tstages = p.stages;
  if (p.stages < 2 && p.tail && fixed + 2 * (per - kTailBytes) + kTailBytes <= kSmemLimit) {
    p.stages = 2;
    p.tstages = 1;
  }
  p.q_off = p.stages * stage;
  p.p_off = p.q_off + p.q_bytes;              // q_bytes is a multiple of 1024
  p.t_off = p.p_off + kChunkBytes;
  p.i_off = p.t_off + p.tail * p.tstages * kTailBytes;
  p.m_off = p.i_off + p.stages * kTile * 8;
  p.smem = p.m_off + p.stages * 8 + kBars * 8 + 8 * C + 2 * C;
  return p;
}

struct AttendTc {
  KvAttendArgs a;
  Plan p;
  int col_groups;
};

__device__ __forceinline__ uint64_t desc128(uint32_t saddr) {     // 128-byte swizzle, 1024-byte groups
  uint64_t d = static_cast<uint64_t>((saddr >> 4) & 0x3FFFu);
  d |= static_cast<uint64_t>(1u) << 16;
  d |= static_cast<uint64_t>(1024u >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(2u) << 61;
  return d;
}
__device__ __forceinline__ uint64_t desc64(uint32_t saddr) {      // 64-byte swizzle, 512-byte groups
  uint64_t d = static_cast<uint64_t>((saddr >> 4) & 0x3FFFu);
  d |= static_cast<uint64_t>(1u) << 16;
  d |= static_cast<uint64_t>(512u >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(4u) << 61;
  return d;
}

// kind::f8f6f4, fp32 accumulators, M = 128: operand types (0 e4m3, 1 e5m2), both operands
// K-major (mn = 0) or both MN-major (mn = 1).
__host__ __device__ constexpr uint32_t idesc(int n, int b_type, int mn) {
  return (1u << 4) | (static_cast<uint32_t>(b_type) << 10) | (static_cast<uint32_t>(mn) << 15) |
         (static_cast<uint32_t>(mn) << 16) | (static_cast<uint32_t>(n >> 3) << 17) |
         (static_cast<uint32_t>(128 >> 4) << 24);
}

#define LSA_R8(r, o) "=r"(r[o]), "=r"(r[o + 1]), "=r"(r[o + 2]), "=r"(r[o + 3]), "=r"(r[o + 4]), "=r"(r[o + 5]), "=r"(r[o + 6]), "=r"(r[o + 7])
#define LSA_I8(r, o) "r"(r[o]), "r"(r[o + 1]), "r"(r[o + 2]), "r"(r[o + 3]), "r"(r[o + 4]), "r"(r[o + 5]), "r"(r[o + 6]), "r"(r[o + 7])

// n columns of this thread's lane (no wait).
__device__ __forceinline__ void tmem_ld(uint32_t t, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];" : LSA_R8(r, 0) : "r"(t));
}
__device__ __forceinline__ void tmem_ld(uint32_t t, uint32_t (&r)[16]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
               "%14, %15}, [%16];" : LSA_R8(r, 0), LSA_R8(r, 8) : "r"(t));
}
__device__ __forceinline__ void tmem_ld(uint32_t t, uint32_t (&r)[32]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
               "%14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
               : LSA_R8(r, 0), LSA_R8(r, 8), LSA_R8(r, 16), LSA_R8(r, 24) : "r"(t));
}
__device__ __forceinline__ void tmem_st(uint32_t t, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::LSA_I8(r, 0), "r"(t) : "memory");
}
__device__ __forceinline__ void tmem_st(uint32_t t, const uint32_t (&r)[16]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, "
               "%13, %14, %15};" ::LSA_I8(r, 0), LSA_I8(r, 8), "r"(t) : "memory");
}
__device__ __forceinline__ void tmem_st(uint32_t t, const uint32_t (&r)[32]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, "
               "%13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};"
               ::LSA_I8(r, 0), LSA_I8(r, 8), LSA_I8(r, 16), LSA_I8(r, 24), "r"(t) : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void group_sync(int id) { asm volatile("barrier.cta.sync %0, 128;" ::"r"(id) : "memory"); }
__device__ __forceinline__ bool group_any(int id, bool v) {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\t"
               "barrier.cta.red.or.pred q, %2, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
               : "=r"(r) : "r"(static_cast<uint32_t>(v)), "r"(id) : "memory");
  return r != 0;
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float lg2(float x) {
  float r;
  asm("lg2.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ int ordered(float x) {                 // order-preserving image of a non-NaN float
  const int i = __float_as_int(x);
  return i >= 0 ? i : i ^ 0x7fffffff;
}
__device__ __forceinline__ float unordered(int i) { return __int_as_float(i >= 0 ? i : i ^ 0x7fffffff); }

// Two weights as their e4m3 codes (low half) and the e5m2 codes of what is left (high half).
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
  const __nv_fp8x2_storage_t h = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const float2 f = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(h, __NV_E4M3)));
  hi = h;
  lo = __nv_cvt_float2_to_fp8x2(make_float2(a - f.x, b - f.y), __NV_SATFINITE, __NV_E5M2);
}

template <int C>
__global__ void __launch_bounds__(kThreads, 1)
kv_attend_tc_kernel(const __grid_constant__ CUtensorMap map, const __grid_constant__ CUtensorMap map_tail,
                    const __grid_constant__ AttendTc t) {
  constexpr int NC = C / 2;                                // columns of a softmax warp
  constexpr uint32_t kO = 4 * C;                           // tensor-memory columns: S (two of 2C), then O^T
  extern __shared__ __align__(1024) uint8_t smem[];
  const KvAttendArgs& a = t.a;
  const Plan& pl = t.p;
  const KvGeom& g = a.g;
  const uint32_t tmem_cols = C == 64 ? 512u : C == 32 ? 256u : 128u;
  uint8_t* ring = smem;
  uint8_t* qimg = smem + pl.q_off;
  uint8_t* pbuf = smem + pl.p_off;
  uint8_t* tails = smem + pl.t_off;
  float2* info = reinterpret_cast<float2*>(smem + pl.i_off);           // [stages][128]: scale, token word
  volatile int* skip = reinterpret_cast<volatile int*>(smem + pl.m_off);        // [stages][2]
  float2* qr = reinterpret_cast<float2*>(smem + pl.m_off + pl.stages * 8);      // [C]: query factor, reference
  uint64_t* bars = reinterpret_cast<uint64_t*>(qr + C);
  uint16_t* qi = reinterpret_cast<uint16_t*>(bars + kBars);               // [C]: query token of a column
  uint64_t* full = bars;                    // [6]
  uint64_t* empty = bars + 6;               // [6]
  uint64_t* tfull = bars + 12;              // [6]
  uint64_t* tempty = bars + 18;             // [6]
  uint64_t* ifull = bars + 24;              // [6]
  uint64_t* sfull = bars + 30;              // [2]
  uint64_t* pfull = bars + 32;
  uint64_t* pdone = bars + 33;
  uint64_t* drain = bars + 34;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 35);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + 36);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int hg = a.H / g.G, ncol = a.Tq * hg;
  int u = blockIdx.x;
  const int cg = u % t.col_groups; u /= t.col_groups;
  const int part = u % a.splits; u /= a.splits;
  const int head = u % g.G, b = u / g.G;
  const int c_base = cg * C, n_c = min(C, ncol - c_base);
  const KvSpan sp = kv_span(a, b);
  const int tiles = (sp.total + kTile - 1) / kTile;
  const int tile0 = static_cast<int>(static_cast<long long>(tiles) * part / a.splits);
  const int n = static_cast<int>(static_cast<long long>(tiles) * (part + 1) / a.splits) - tile0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < pl.stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
      mbar_init(&tfull[s], 1);
      mbar_init(&tempty[s], 1);
      mbar_init(&ifull[s], 32);
    }
    mbar_init(&sfull[0], 1);
    mbar_init(&sfull[1], 1);
    mbar_init(pfull, 8);
    mbar_init(pdone, 1);
    mbar_init(drain, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) tmem_alloc(tmem_slot, tmem_cols);
  // The query image: row c the first terms of column c, row C + c the second ones.  The
  // rows of missing columns and the elements past d are zeros.
  {
    const int n_kf = pl.n_k - pl.tail, dpad = pl.ksteps * 32;
    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q);
    for (int c = warp; c < C; c += kThreads / 32) {
      const int col = c_base + c;
      const bool real = c < n_c;
      const int i = real ? col / hg : 0;
      const __nv_bfloat16* row = q + ((static_cast<size_t>(b) * a.Tq + i) * a.H + head * hg + (real ? col - i * hg : 0)) * a.d;
      uint4 v[3];                                          // d <= 576: at most 72 groups of 8
      uint32_t m = 0;
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        const int e = (lane + 32 * k) * 8;
        v[k] = make_uint4(0, 0, 0, 0);
        if (real && e < a.d) v[k] = __ldg(reinterpret_cast<const uint4*>(row + e));
        const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
        for (int x = 0; x < 4; ++x) m = max(m, max((w[x] << 16) & 0x7fffffffu, w[x] & 0x7fff0000u));
      }
      m = __reduce_max_sync(0xffffffffu, m);
      const bool finite = m < 0x7f800000u;
      // s = 2^e, the smallest (from 2^-100) with max|q| / s <= 448
      const int se = max(static_cast<int>(m >> 23) - 8 + ((m & 0x7fffffu) > 0x600000u ? 1 : 0), 27);
      const float inv = finite ? __uint_as_float(static_cast<uint32_t>(254 - se) << 23) : 0.f;
      if (lane == 0) {
        const float s = finite ? __uint_as_float(static_cast<uint32_t>(se) << 23) : __uint_as_float(0x7fc00000u);
        qr[c] = make_float2(real ? s * a.sm * 1.44269504088896f : 0.f, kUnset);
        qi[c] = static_cast<uint16_t>(i);
      }
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        const int e = (lane + 32 * k) * 8;
        if (e >= dpad) continue;
        const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const float f0 = __uint_as_float(w[x] << 16) * inv, f1 = __uint_as_float(w[x] & 0xffff0000u) * inv;
          hi[x] = __nv_cvt_float2_to_fp8x2(make_float2(f0, f1), __NV_SATFINITE, __NV_E4M3);
          const float2 h = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(hi[x]), __NV_E4M3)));
          lo[x] = __nv_cvt_float2_to_fp8x2(make_float2(f0 - h.x, f1 - h.y), __NV_SATFINITE, __NV_E4M3);
        }
        const uint2 hv = make_uint2(hi[0] | (hi[1] << 16), hi[2] | (hi[3] << 16));
        const uint2 lv = make_uint2(lo[0] | (lo[1] << 16), lo[2] | (lo[3] << 16));
        const int chunk = e / 128, j = (e % 128) / 16, x = e % 16, rl = C + c;
        if (chunk < n_kf) {
          uint8_t* base = qimg + chunk * (2 * C * 128);
          *reinterpret_cast<uint2*>(base + c * 128 + ((j ^ (c & 7)) * 16) + x) = hv;
          *reinterpret_cast<uint2*>(base + rl * 128 + ((j ^ (rl & 7)) * 16) + x) = lv;
        } else {
          uint8_t* base = qimg + n_kf * (2 * C * 128);
          *reinterpret_cast<uint2*>(base + c * 64 + ((j ^ ((c >> 1) & 3)) * 16) + x) = hv;
          *reinterpret_cast<uint2*>(base + rl * 64 + ((j ^ ((rl >> 1) & 3)) * 16) + x) = lv;
        }
      }
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    // ---------------------------------------------------------------- producer
    uint64_t policy;
    asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(policy));
    const int p_first = sp.len - a.Tq + (c_base / hg), p_last = sp.len - a.Tq + (c_base + n_c - 1) / hg;
    int rows[4], words[4];
    float scales[4];
    auto resolve = [&](int tile) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int v = tile * kTile + 4 * lane + e;
        bool main = false;
        int tok = v < sp.total ? kv_token(a, sp, b, v, main) : -1;
        rows[e] = -1;
        scales[e] = 0.f;
        words[e] = 0;
        if (tok < 0) continue;
        const bool sees0 = kv_sees(a, tok, p_first), sees1 = kv_sees(a, tok, p_last);
        if (p_first == p_last && sees0 != main) continue;   // outside the one query's set, or a list entry inside it
        const long long row = kv_row(g, b, tok);
        if (row < 0) {
          raise_status(a.status, LSA_ERR_RANGE);
          continue;
        }
        rows[e] = static_cast<int>(row * g.G + head);
        scales[e] = __ldg(g.scale + kv_scale_at(g, b, tok, head));
        // A main token is seen by every query between two that see it; a list entry by all when it
        // lies behind every query or before every window.
        const bool all = p_first == p_last ||
                         (main ? sees0 && sees1
                               : tok > p_last || (tok >= a.sinks && a.window >= 0 && tok <= static_cast<long long>(p_first) - a.window));
        words[e] = tok | (main ? 0 : kListFlag) | (all ? kAllFlag : 0);
      }
    };
    const uint32_t bytes = static_cast<uint32_t>(pl.n_full) * kChunkBytes;
    const int n_kf = pl.n_k - pl.tail, ex0 = max(pl.v0, n_kf);
    bool ok = true;
    int s = 0, ts = 0, issued = 0;
    uint32_t ph = 0, tph = 0;
    if (n > 0) resolve(tile0);
    for (int j = 0; j < n; ++j) {
      const unsigned have = __ballot_sync(0xffffffffu, rows[0] >= 0 || rows[1] >= 0 || rows[2] >= 0 || rows[3] >= 0);
      int any = rows[0] >= 0 ? rows[0] : rows[1] >= 0 ? rows[1] : rows[2] >= 0 ? rows[2] : rows[3];
      any = __shfl_sync(0xffffffffu, any, have ? __ffs(have) - 1 : 0);  // a row for the places without one
      if (lane == 0) {
        ok = mbar_wait(&empty[s], ph ^ 1, abort_flag);
        if (ok && pl.tail) ok = mbar_wait(&tempty[ts], tph ^ 1, abort_flag);
        if (ok) {
          skip[2 * s] = have == 0;
          if (have) {
            mbar_expect_tx(&full[s], bytes);
            if (pl.tail) mbar_expect_tx(&tfull[ts], kTailBytes);
          } else {
            mbar_arrive(&full[s]);
            if (pl.tail) mbar_arrive(&tfull[ts]);
          }
        }
      }
      ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
      if (!ok) break;
      if (have) {
        int r[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) r[e] = rows[e] >= 0 ? rows[e] : any;
        uint8_t* dst = ring + static_cast<size_t>(s) * bytes + lane * 512;
        for (int c = 0; c < n_kf; ++c)
          tma_gather4_2d(dst + c * kChunkBytes, &map, c * 128, r[0], r[1], r[2], r[3], &full[s], policy);
        for (int c = ex0; c < pl.v0 + pl.n_v; ++c)
          tma_gather4_2d(dst + (n_kf + c - ex0) * kChunkBytes, &map, c * 128, r[0], r[1], r[2], r[3], &full[s], policy);
        if (pl.tail)
          tma_gather4_2d(tails + ts * kTailBytes + lane * 256, &map_tail, n_kf * 128, r[0], r[1], r[2], r[3],
                         &tfull[ts], policy);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) info[s * kTile + 4 * lane + e] = make_float2(scales[e], __int_as_float(words[e]));
      mbar_arrive(&ifull[s]);
      ++issued;
      if (++s == pl.stages) { s = 0; ph ^= 1; }
      if (++ts == pl.tstages) { ts = 0; tph ^= 1; }
      if (j + 1 < n) resolve(tile0 + j + 1);
    }
    if (lane == 0) {
      // every copy this warp issued has landed before the block exits
      volatile int no_abort = 0;
      for (int k = max(0, issued - pl.stages); k < issued; ++k)
        if (!mbar_wait(&full[k % pl.stages], (k / pl.stages) & 1, &no_abort)) break;
      if (pl.tail)
        for (int k = max(0, issued - pl.tstages); k < issued; ++k)
          if (!mbar_wait(&tfull[k % pl.tstages], (k / pl.tstages) & 1, &no_abort)) break;
    }
  } else if (warp == 1 && lane == 0) {
    // ---------------------------------------------------------------- MMA issuer
    const uint32_t ring_u = smem_u32(ring), q_u = smem_u32(qimg), p_u = smem_u32(pbuf), tail_u = smem_u32(tails);
    const uint32_t stage_b = static_cast<uint32_t>(pl.n_full) * kChunkBytes;
    const int n_kf = pl.n_k - pl.tail;
    constexpr uint32_t id_s = idesc(2 * C, 0, 0), id_hi = idesc(C, 0, 1), id_lo = idesc(C, 1, 1);
    int s = 0, ts = 0;
    uint32_t ph = 0, tph = 0;
    auto scores = [&](int j) -> bool {
      if (!mbar_wait(&full[s], ph, abort_flag)) return false;
      if (pl.tail && !mbar_wait(&tfull[ts], tph, abort_flag)) return false;
      tc_fence_after();
      if (!skip[2 * s]) {
        const uint32_t d_t = tmem + (j & 1) * (2 * C);
        for (int ks = 0; ks < pl.ksteps; ++ks) {
          const int chunk = ks >> 2;
          uint64_t ad, bd;
          if (chunk < n_kf) {
            ad = desc128(ring_u + s * stage_b + chunk * kChunkBytes) + (ks & 3) * 2;
            bd = desc128(q_u + chunk * (2 * C * 128)) + (ks & 3) * 2;
          } else {
            ad = desc64(tail_u + ts * kTailBytes) + (ks & 3) * 2;
            bd = desc64(q_u + n_kf * (2 * C * 128)) + (ks & 3) * 2;
          }
          mma<true>(d_t, ad, bd, id_s, ks > 0 ? 1u : 0u);
        }
      }
      mma_commit(&sfull[j & 1]);
      if (pl.tail) mma_commit(&tempty[ts]);
      if (++s == pl.stages) { s = 0; ph ^= 1; }
      if (++ts == pl.tstages) { ts = 0; tph ^= 1; }
      return true;
    };
    bool ok = n > 0 ? scores(0) : true;
    uint32_t acc = 0;
    int vs = 0;
    for (int j = 0; ok && j < n; ++j) {
      if (j + 1 < n && !(ok = scores(j + 1))) break;
      if (!(ok = mbar_wait(pfull, j & 1, abort_flag))) break;
      tc_fence_after();
      if (!skip[2 * vs]) {
        for (int m = 0; m < pl.n_v; ++m) {
          const uint64_t ad = desc128(ring_u + vs * stage_b + plan_v_slot(pl, pl.v0 + m) * kChunkBytes);
          const uint64_t bd = desc128(p_u);
#pragma unroll
          for (int ks = 0; ks < 4; ++ks) {
            mma<true>(tmem + kO + m * C, ad + ks * 256, bd + ks * 256, id_hi, acc | (ks > 0 ? 1u : 0u));
            mma<true>(tmem + kO + m * C, ad + ks * 256, bd + ks * 256 + 4, id_lo, 1u);
          }
        }
        acc = 1;
      }
      mma_commit(&empty[vs]);
      mma_commit(pdone);
      if (++vs == pl.stages) vs = 0;
    }
    mma_commit(drain);
    volatile int no_abort = 0;
    mbar_wait(drain, 0, &no_abort);
  } else if (warp >= 4) {
    // ---------------------------------------------------------------- weights and results
    const int wg = (warp - 4) >> 2, quad = warp & 3, row = quad * 32 + lane;
    const int c0 = wg * NC, bar_id = 1 + wg;
    const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
    // Scratch of 256 words for the group, in its own columns' bytes of the weights buffer (two
    // words a row), while no MMA reads them.
    auto scratch = [&](int i) {
      const int r = i >> 1;
      return reinterpret_cast<int*>(pbuf + r * 128 + (((c0 >> 4) ^ (r & 7)) * 16) + (c0 & 15) + (i & 1) * 4);
    };
    float l[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) l[c] = 0.f;
    bool ok = true, have_o = false;
    int s = 0;
    uint32_t ph = 0;
    for (int j = 0; j < n; ++j) {
      if (ok) ok = mbar_wait(&ifull[s], ph, abort_flag);
      if (ok) ok = mbar_wait(&sfull[j & 1], (j >> 1) & 1, abort_flag);
      tc_fence_after();
      const bool empty_tile = ok && skip[2 * s] != 0;
      float y[NC];
      float scale = 0.f;
      bool over = !ok;
      if (!empty_tile) {
        uint32_t hi[NC], lo[NC];
        const uint32_t st = tmem + lanes + (j & 1) * (2 * C) + c0;
        tmem_ld(st, hi);
        tmem_ld(st + C, lo);
        const float2 in = info[s * kTile + row];
        scale = in.x;
        const int word = __float_as_int(in.y);
        // an unseen token has scale 0: y = 0 + log2(0) = -infinity
        const float ls = scale == 0.f ? -INFINITY : lg2(scale);
        tmem_wait_ld();
        const bool masks = a.Tq > 1 && !__all_sync(0xffffffffu, word < 0 || scale == 0.f);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          const float2 f = qr[c0 + c];
          const float x = (__uint_as_float(hi[c]) + __uint_as_float(lo[c])) * scale;
          y[c] = fmaf(x, f.x, ls);
          if (masks) {
            const int p = sp.len - a.Tq + qi[c0 + c];
            const bool in_main = kv_sees(a, word & (kListFlag - 1), p);
            if (word >= 0 && ((word & kListFlag) ? in_main : !in_main)) y[c] = -INFINITY;
          }
          over |= y[c] - f.y > kLimit;
        }
      }
      if (group_any(bar_id, over)) {
        if (group_any(bar_id, !ok)) break;                 // uniform in the group
        if (!empty_tile) {
          // The weights buffer is scratch once the MMAs that read it are done.
          if (j > 0) ok = mbar_wait(pdone, (j - 1) & 1, abort_flag);
          tc_fence_after();
          int mine = ordered(kUnset);
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            const float v = y[c] == y[c] ? fmaxf(y[c], kUnset) : kUnset;    // a NaN does not move the reference
            const int m = __reduce_max_sync(0xffffffffu, ordered(v));
            if (lane == c) mine = m;
          }
          if (lane < NC) *scratch(quad * 32 + lane) = mine;
          group_sync(bar_id);
          float old = kUnset, now = kUnset;
          if (lane < NC) {
            old = qr[c0 + lane].y;
            const float m = unordered(max(max(*scratch(lane), *scratch(32 + lane)), max(*scratch(64 + lane), *scratch(96 + lane))));
            now = m - old > kLimit ? m - kTarget : old;
          }
          const float f_mine = ex2(old - now);             // 0 from unset
          group_sync(bar_id);                              // every warp has read the old reference
          if (quad == 0 && lane < NC) qr[c0 + lane].y = now;
          group_sync(bar_id);
#pragma unroll
          for (int c = 0; c < NC; ++c) l[c] *= __shfl_sync(0xffffffffu, f_mine, c);
          if (have_o) {
            for (int m = 0; m < pl.n_v; ++m) {
              uint32_t o[NC];
              const uint32_t at = tmem + lanes + kO + m * C + c0;
              tmem_ld(at, o);
              tmem_wait_ld();
#pragma unroll
              for (int c = 0; c < NC; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * __shfl_sync(0xffffffffu, f_mine, c));
              tmem_st(at, o);
            }
            tmem_wait_st();
          }
        }
      }
      if (ok && j > 0) ok = mbar_wait(pdone, (j - 1) & 1, abort_flag);
      if (!empty_tile) {
        // Of a NaN scale only the columns that see the token become NaN.
        const float inv = scale > 0.f ? 1.0f / scale : 1.0f;
        uint32_t hi[NC / 4], lo[NC / 4];
#pragma unroll
        for (int c = 0; c < NC; c += 4) {
          float p[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            p[e] = ex2(y[c + e] - qr[c0 + c + e].y);
            l[c + e] = fmaf(p[e], inv, l[c + e]);
          }
          uint32_t h0, h1, l0, l1;
          split2(p[0], p[1], h0, l0);
          split2(p[2], p[3], h1, l1);
          hi[c / 4] = h0 | (h1 << 16);
          lo[c / 4] = l0 | (l1 << 16);
        }
        uint8_t* pr = pbuf + row * 128;
        if constexpr (NC >= 16) {
#pragma unroll
          for (int k = 0; k < NC / 16; ++k) {
            const int ch = c0 / 16 + k, cl = 4 + ch;
            *reinterpret_cast<uint4*>(pr + ((ch ^ (row & 7)) * 16)) = make_uint4(hi[4 * k], hi[4 * k + 1], hi[4 * k + 2], hi[4 * k + 3]);
            *reinterpret_cast<uint4*>(pr + ((cl ^ (row & 7)) * 16)) = make_uint4(lo[4 * k], lo[4 * k + 1], lo[4 * k + 2], lo[4 * k + 3]);
          }
        } else {
          *reinterpret_cast<uint2*>(pr + ((0 ^ (row & 7)) * 16) + c0) = make_uint2(hi[0], hi[1]);
          *reinterpret_cast<uint2*>(pr + ((4 ^ (row & 7)) * 16) + c0) = make_uint2(lo[0], lo[1]);
        }
        have_o = true;
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(pfull);
      if (++s == pl.stages) { s = 0; ph ^= 1; }
    }
    // the last tile's values are in; sums over the block's tokens
    if (ok && n > 0) ok = mbar_wait(pdone, (n - 1) & 1, abort_flag);
    tc_fence_after();
    const bool fail_any = group_any(bar_id, !ok);
    float mine = 0.f;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      float v = l[c];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      if (lane == c) mine = v;
    }
    if (lane < NC) *scratch(quad * 32 + lane) = __float_as_int(mine);
    group_sync(bar_id);
    float tot = 0.f, ref = kUnset;
    if (lane < NC) {
      auto part_sum = [&](int i) { return __int_as_float(*scratch(i)); };
      tot = (part_sum(lane) + part_sum(32 + lane)) + (part_sum(64 + lane) + part_sum(96 + lane));
      ref = qr[c0 + lane].y;
    }
    const bool direct = a.splits == 1;
    const size_t part_at = ((static_cast<size_t>(b) * g.G + head) * a.splits + part) * ncol + c_base + c0;
    if (quad == 0 && lane < NC && c0 + lane < n_c && !fail_any) {
      if (direct) {
        const int col = c_base + c0 + lane;
        const size_t oc = (static_cast<size_t>(b) * a.Tq + col / hg) * a.H + head * hg + col % hg;
        if (a.lse) a.lse[oc] = tot == 0.f ? -INFINITY : (ref + log2f(tot)) * 0.693147180559945f;
      } else {
        a.part_m[part_at + lane] = ref;
        a.part_l[part_at + lane] = tot;
      }
    }
    if (!fail_any) {
      const float rinv = direct ? (tot == 0.f ? 0.f : 1.0f / tot) : 1.f;
      for (int m = 0; m < pl.n_v; ++m) {
        const int vc = (pl.v0 + m) * 128 + row - a.voff;   // value column of this lane
        uint32_t o[NC];
        if (have_o) {
          tmem_ld(tmem + lanes + kO + m * C + c0, o);
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int c = 0; c < NC; ++c) o[c] = 0u;
        }
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          const float r = __shfl_sync(0xffffffffu, rinv, c);
          if (c0 + c >= n_c || vc < 0 || vc >= a.dv) continue;
          const float v = __uint_as_float(o[c]);
          if (direct) {
            const int col = c_base + c0 + c;
            const size_t oc = (static_cast<size_t>(b) * a.Tq + col / hg) * a.H + head * hg + col % hg;
            static_cast<__nv_bfloat16*>(a.out)[oc * a.dv + vc] = __float2bfloat16_rn(r == 0.f ? 0.f : v * r);
          } else {
            a.part_o[(part_at + c) * a.dv + vc] = v;
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && *abort_flag) raise_status(a.status, LSA_ERR_TIMEOUT);
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, tmem_cols);
  }
}

int columns(int ncol) { return ncol <= 16 ? 16 : ncol <= 32 ? 32 : 64; }

template <int C>
int launch_c(const CUtensorMap& map, const CUtensorMap& tail, const AttendTc& t, long long grid, cudaStream_t s) {
  const cudaError_t e = cudaFuncSetAttribute(kv_attend_tc_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, t.p.smem);
  if (e != cudaSuccess) return fail(LSA_ERR_CUDA, "kv_attend: %s", cudaGetErrorString(e));
  kv_attend_tc_kernel<C><<<static_cast<unsigned>(grid), kThreads, t.p.smem, s>>>(map, tail, t);
  return check_launch("kv_attend");
}

}  // namespace

bool kv_attend_tc_supported(int N, int d, int dv, int voff, int qdt, int ncol) {
  if (qdt != LSA_BF16 || d % 8 != 0 || d > 576 || N > (1 << 30)) return false;
  const Plan p = make_plan(d, dv, voff, columns(ncol));
  return p.n_v <= 4 && p.stages >= 2 && p.smem <= kSmemLimit;
}

int kv_attend_splits_tc(int B, int G, int ncol, long long max_tokens) {
  const int C = columns(ncol);
  const long long units = static_cast<long long>(B) * G * ((ncol + C - 1) / C);
  const long long tiles = std::max<long long>(1, (max_tokens + kTile - 1) / kTile);
  const long long least = (max_tokens + 16383) / 16384;   // the weights' range (see the top)
  // One block per SM: the split with the fewest tile times, a block's start and end counted
  // as four tiles.
  long long best = std::max<long long>(1, least), cost = -1;
  for (long long s = best; s <= std::max<long long>(best, std::min<long long>(tiles, 256)); ++s) {
    const long long waves = (units * s + 147) / 148, c = waves * ((tiles + s - 1) / s + 4);
    if (cost < 0 || c < cost) {
      cost = c;
      best = s;
    }
    if (waves > 16 && s > best + 16) break;
  }
  return static_cast<int>(best);
}

int launch_kv_attend_tc(const KvAttendArgs& a, cudaStream_t s) {
  const int ncol = a.Tq * (a.H / a.g.G), C = columns(ncol);
  AttendTc t{};
  t.a = a;
  t.p = make_plan(a.d, a.dv, a.voff, C);
  t.col_groups = (ncol + C - 1) / C;
  EncodeTiledFn enc = encode_fn();
  if (!enc) return fail(LSA_ERR_CUDA, "kv_attend: cuTensorMapEncodeTiled unavailable");
  CUtensorMap map, tail;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(a.g.W),
                              (static_cast<cuuint64_t>(a.g.pages) << a.g.page_log) * static_cast<cuuint64_t>(a.g.G)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(a.g.W)};
  const cuuint32_t estr[2] = {1, 1}, box[2] = {128, 1}, box_tail[2] = {64, 1};
  CUresult cr = enc(&map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, a.g.rows, dims, strides, box, estr,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (cr == CUDA_SUCCESS)
    cr = enc(&tail, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, a.g.rows, dims, strides, box_tail, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (cr != CUDA_SUCCESS) return fail(LSA_ERR_CUDA, "kv_attend: tensor map encode failed (%d)", static_cast<int>(cr));
  const long long grid = static_cast<long long>(a.g.B) * a.g.G * a.splits * t.col_groups;
  if (C == 64) return launch_c<64>(map, tail, t, grid, s);
  if (C == 32) return launch_c<32>(map, tail, t, grid, s);
  return launch_c<16>(map, tail, t, grid, s);
}

}  // namespace lsa
