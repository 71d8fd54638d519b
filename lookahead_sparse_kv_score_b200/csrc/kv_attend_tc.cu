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
// 2^-17.  The reference weight is 2^k with k = log2(tokens of the part) - 8 (0 to 6, parts
// of at most 16384 tokens), so the weights lost below the range are less than 2^-9 of the sum.
// Scores, the sum of the weights and the accumulators are fp32.
//
// Scales.  y_tc = sm log2(e) scale_t (q_c . k_t) + log2(scale_t); the value weight is
// P''_tc = 2^(y_tc - r_c) and the softmax weight P''_tc / scale_t, so one exponential serves
// both sums and the scale never multiplies the codes.  r_c is set so that the largest weight
// seen is 2^k and kept until a weight would pass 448: then the block's O^T columns are
// multiplied by 2^(r_old - r_new) in tensor memory.  That is rare after the first tile, so the
// cross-lane maxima are only computed then; otherwise a tile costs one vote.
//
// Roles (13 warps; 9 with 16 columns): warps 0-3 bring the rows, one token a lane, chunk by
// chunk, and write the tokens' scales; warps 4-11 hold one token a lane and half of the
// columns each; the last warp issues the MMAs, S a tile ahead of O, a chunk at a time as chunks
// arrive.  A warp whose 32 rows follow one another in memory (a dense cache, pages of 16 and
// more) brings them as TMA boxes; other rows (a fetched list) go by 16-byte asynchronous
// copies in the MMA's swizzle, with zeros where a place has no token.  TMA row gathers were
// slower: 65 clocks a four-row instruction, 8 bytes a clock and SM, a third of the HBM rate.
//
// A sequence's tokens are divided among the blocks of a cluster (and, when there are few
// sequences, among several clusters).  At the end each block lays its O^T and sums in its
// shared memory, and the blocks of the cluster join a share of the columns each, reading
// one another's: no partial sums cross memory unless there is more than one cluster.
//
// Waits are bounded; on expiry LSA_ERR_TIMEOUT is raised, MMAs and copies in flight are drained
// and the tensor memory is freed.
#include <cuda.h>

#include <algorithm>
#include <climits>
#include <type_traits>

#include "kv_common.cuh"
#include "tc_ptx.cuh"

namespace lsa {
namespace {

using namespace tc;

constexpr int kTile = 128;
constexpr int kProducers = 128;               // warps 0-3

// A block's shape by its query columns.  With 64 columns two groups of four warps hold half of
// them each; with 16 one group holds all, and two blocks share an SM.
template <int C>
struct Shape {
  static constexpr int kGroups = C == 16 ? 1 : 2;
  static constexpr int NC = C / kGroups;                   // columns of a weights warp
  static constexpr int kWeights = 4 * kGroups;             // warps
  static constexpr int kMmaWarp = 4 + kWeights;
  static constexpr int kThreads = 32 * (kMmaWarp + 1);
  static constexpr int kBlocks = C == 64 ? 1 : 2;          // blocks an SM, where shared memory allows
  static constexpr uint32_t kTmemCols = C == 64 ? 512 : C == 32 ? 256 : 128;
};
constexpr int kSmemLimit = 227 * 1024;
constexpr int kChunkBytes = kTile * 128;      // 128 columns of a tile, 128-byte swizzle
constexpr int kTailBytes = kTile * 64;        // the last 64 key columns, 64-byte swizzle
constexpr int kMaxStages = 4;
constexpr int kMaxSlots = 12;                 // stages times 128-column chunks: 16 KB each
constexpr int kBars = 46;                     // 8-byte words of barriers and flags
constexpr float kUnset = 3.0e38f;             // minus the reference exponent before any token was seen
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
  int q_off, p_off, t_off, i_off, m_off, smem;
};

__host__ __device__ inline int plan_v_slot(const Plan& p, int chunk) {   // ring slot of a value chunk
  const int n_kf = p.n_k - p.tail;
  if (chunk < n_kf) return chunk;
  return n_kf + chunk - (p.v0 > n_kf ? p.v0 : n_kf);
}

// limit: shared memory of a block.
Plan make_plan(int d, int dv, int voff, int C, int limit) {
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
  const int q_bytes = 2 * C * (n_kf * 128 + p.tail * 64);     // a multiple of 1024
  const int stage = p.n_full * kChunkBytes;
  const int fixed = q_bytes + kChunkBytes /* weights */ + kBars * 8 + C * (8 + 2);
  // whole stages with their tails while they fit, else two stages on one tail
  const int per = stage + p.tail * kTailBytes + kTile * 8;
  p.stages = std::min({kMaxStages, (limit - fixed) / per, kMaxSlots / p.n_full});
  p.tstages = p.stages;
  if (p.stages < 2 && p.tail && fixed + 2 * (per - kTailBytes) + kTailBytes <= limit) {
    p.stages = 2;
    p.tstages = 1;
  }
  p.q_off = p.stages * stage;
  p.p_off = p.q_off + q_bytes;
  p.t_off = p.p_off + kChunkBytes;
  p.i_off = p.t_off + p.tail * p.tstages * kTailBytes;
  p.m_off = p.i_off + p.stages * kTile * 8;
  p.smem = p.m_off + kBars * 8 + C * (8 + 2);
  return p;
}

struct AttendTc {
  KvAttendArgs a;
  Plan p;
  int col_groups, cluster;
  int run;          // rows of a TMA box (16 or 32 places whose rows follow one another), 0: no maps
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
__device__ __forceinline__ void tmem_ld(uint32_t t, uint32_t (&r)[16]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
               "%14, %15}, [%16];" : LSA_R8(r, 0), LSA_R8(r, 8) : "r"(t));
}
__device__ __forceinline__ void tmem_ld(uint32_t t, uint32_t (&r)[32]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
               "%14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
               : LSA_R8(r, 0), LSA_R8(r, 8), LSA_R8(r, 16), LSA_R8(r, 24) : "r"(t));
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
// Two fp32 operations an instruction, each rounded as the single one.
__device__ __forceinline__ float2 pair(uint32_t a, uint32_t b) { return make_float2(__uint_as_float(a), __uint_as_float(b)); }
__device__ __forceinline__ unsigned long long bits2(float2 a) {
  return (static_cast<unsigned long long>(__float_as_uint(a.y)) << 32) | __float_as_uint(a.x);
}
__device__ __forceinline__ float2 from2(unsigned long long a) {
  return make_float2(__uint_as_float(static_cast<uint32_t>(a)), __uint_as_float(static_cast<uint32_t>(a >> 32)));
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  unsigned long long r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)));
  return from2(r);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  unsigned long long r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)));
  return from2(r);
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  unsigned long long r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)), "l"(bits2(c)));
  return from2(r);
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
__device__ __forceinline__ float warp_max(float x) {               // NaN is ignored
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}

// 16 bytes of global memory to shared memory, or zeros when bytes = 0.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
// Arrives at the barrier when this thread's copies so far have landed.
__device__ __forceinline__ void copies_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// Adds to the bytes a barrier's phase waits for, without arriving.
__device__ __forceinline__ void expect_bytes(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}
__device__ __forceinline__ uint64_t normal_policy() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
  return p;
}
// After an abort the barriers of boxes in flight may never complete: a millisecond, far above
// a copy's time, before the block's shared memory is given up.
__device__ __noinline__ void drain_boxes() {
  const unsigned long long t0 = global_timer();
  while (global_timer() - t0 < 1000000ull) __nanosleep(1000);
}

__device__ __forceinline__ uint32_t peer(uint32_t addr, int rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ float4 peer_ld4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float peer_ld(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
// All threads of the cluster: writes before are seen by reads behind it.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Two weights as their e4m3 codes (low half) and the e5m2 codes of what is left (high half).
__device__ __forceinline__ void split2(float2 p, uint32_t& hi, uint32_t& lo) {
  const __nv_fp8x2_storage_t h = __nv_cvt_float2_to_fp8x2(p, __NV_SATFINITE, __NV_E4M3);
  const float2 f = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(h, __NV_E4M3)));
  hi = h;
  lo = __nv_cvt_float2_to_fp8x2(make_float2(p.x - f.x, p.y - f.y), __NV_SATFINITE, __NV_E5M2);
}

// Blocks of a unit: rank (fastest), column group, cluster of the unit's parts, KV head, sequence.
template <int C>
__global__ void __launch_bounds__(Shape<C>::kThreads, Shape<C>::kBlocks)
kv_attend_tc_kernel(const __grid_constant__ CUtensorMap map, const __grid_constant__ CUtensorMap map_tail,
                    const __grid_constant__ AttendTc t) {
  using Sh = Shape<C>;
  constexpr int NC = Sh::NC, kMmaWarp = Sh::kMmaWarp, kThreads = Sh::kThreads;
  constexpr uint32_t kO = 4 * C;                           // tensor-memory columns: S (two of 2C), then O^T
  constexpr uint32_t kTmemCols = Sh::kTmemCols;
  extern __shared__ __align__(1024) uint8_t smem[];
  const KvAttendArgs& a = t.a;
  const Plan& pl = t.p;
  const KvGeom& g = a.g;
  uint8_t* ring = smem;
  uint8_t* qimg = smem + pl.q_off;
  uint8_t* pbuf = smem + pl.p_off;
  uint8_t* tails = smem + pl.t_off;
  float2* info = reinterpret_cast<float2*>(smem + pl.i_off);           // [stages][128]: scale, token word
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + pl.m_off);
  float* qf = reinterpret_cast<float*>(bars + kBars);                  // [C]: query factor; at the end, sum of weights
  float* nref = qf + C;                                                // [C]: minus the reference exponent
  uint16_t* qi = reinterpret_cast<uint16_t*>(nref + C);                // [C]: query token of a column
  uint64_t* full = bars;                    // [12] by chunk slot
  uint64_t* empty = bars + 12;              // [12]
  uint64_t* tfull = bars + 24;              // [4] tails
  uint64_t* tempty = bars + 28;             // [4]
  uint64_t* ifull = bars + 32;              // [4] token words
  uint64_t* sfull = bars + 36;              // [2]
  uint64_t* pfull = bars + 38;
  uint64_t* pdone = bars + 39;
  uint64_t* qfull = bars + 40;
  uint64_t* drain = bars + 41;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 42);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + 43);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int hg = a.H / g.G, ncol = a.Tq * hg;
  int u = blockIdx.x;
  const int rank = u % t.cluster; u /= t.cluster;
  const int cg = u % t.col_groups; u /= t.col_groups;
  const int grp = u % a.splits; u /= a.splits;             // a.splits: clusters of a unit
  const int head = u % g.G, b = u / g.G;
  const int c_base = cg * C, n_c = min(C, ncol - c_base);
  const KvSpan sp = kv_span(a, b);
  const int tiles = (sp.total + kTile - 1) / kTile;
  const int parts = a.splits * t.cluster, part = grp * t.cluster + rank;
  const int tile0 = static_cast<int>(static_cast<long long>(tiles) * part / parts);
  const int n = static_cast<int>(static_cast<long long>(tiles) * (part + 1) / parts) - tile0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < pl.stages * pl.n_full; ++s) {
      mbar_init(&full[s], kProducers);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < pl.stages; ++s) {
      mbar_init(&tfull[s], kProducers);
      mbar_init(&tempty[s], 1);
      mbar_init(&ifull[s], kProducers);
    }
    mbar_init(&sfull[0], 1);
    mbar_init(&sfull[1], 1);
    mbar_init(pfull, Sh::kWeights);
    mbar_init(pdone, 1);
    mbar_init(qfull, Sh::kWeights);
    mbar_init(drain, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kMmaWarp) tmem_alloc(tmem_slot, kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp < 4) {
    // ---------------------------------------------------------------- producers
    const int p_first = sp.len - a.Tq + (c_base / hg), p_last = sp.len - a.Tq + (c_base + n_c - 1) / hg;
    const int n_kf = pl.n_k - pl.tail, gap = max(pl.v0 - n_kf, 0);   // chunks between keys and values are not read
    const size_t row_bytes = static_cast<size_t>(g.G) * g.W;
    const uint64_t policy = normal_policy();
    // A token takes three dependent loads (list, table, scale beside the row): each is issued
    // a tile ahead of the next.  tok: the tile behind the next; page, scale: the next tile.
    auto load_token = [&](int j, bool& main) -> int {
      const int v = (tile0 + j) * kTile + threadIdx.x;
      main = false;
      return j < n && v < sp.total ? kv_token(a, sp, b, v, main) : -1;
    };
    int tok1, tok2, page1, row = -1, word = 0;              // row: of the pool, without the head
    bool main1, main2;
    float scale = 0.f, scale1;
    auto load_place = [&](int tok, int& page, float& sc) {
      page = -1;
      sc = 0.f;
      if (tok < 0) return;
      page = g.table != nullptr ? __ldg(g.table + static_cast<size_t>(b) * g.n_pages + (tok >> g.page_log)) : tok >> g.page_log;
      sc = __ldg(g.scale + kv_scale_at(g, b, tok, head));
    };
    // The token's row (-1: nothing to read), scale (0: nobody sees it) and word.
    auto settle = [&](int tok, bool main, int page, float sc) {
      row = -1;
      scale = 0.f;
      word = 0;
      if (tok < 0) return;
      const bool sees0 = kv_sees(a, tok, p_first), sees1 = kv_sees(a, tok, p_last);
      if (p_first == p_last && sees0 != main) return;      // outside the one query's set, or a list entry inside it
      const long long phys = static_cast<long long>(b) * g.seq_pages + page;
      if (page < 0 || (g.seq_pages > 0 && page >= g.seq_pages) || phys >= g.pages) {
        raise_status(a.status, LSA_ERR_RANGE);
        return;
      }
      row = static_cast<int>((phys << g.page_log) + (tok & ((1 << g.page_log) - 1)));
      scale = sc;
      // A main token is seen by every query between two that see it; a list entry by all when it
      // lies behind every query or before every window.
      const bool all = p_first == p_last ||
                       (main ? sees0 && sees1
                             : tok > p_last || (tok >= a.sinks && a.window >= 0 && tok <= static_cast<long long>(p_first) - a.window));
      word = tok | (main ? 0 : kListFlag) | (all ? kAllFlag : 0);
    };
    tok1 = load_token(0, main1);
    tok2 = load_token(1, main2);
    load_place(tok1, page1, scale1);
    int s = 0, ts = 0;
    uint32_t ph = 0, tph = 0;
    bool ok = true;
    for (int j = 0; j < n; ++j) {
      int page2;
      float scale2;
      bool main3;
      load_place(tok2, page2, scale2);
      const int tok3 = load_token(j + 2, main3);
      settle(tok1, main1, page1, scale1);
      // whether the warp's rows are runs of t.run rows, for the TMA
      const int in_run = t.run > 0 ? lane & (t.run - 1) : 0, run_first = __shfl_sync(0xffffffffu, row, lane - in_run);
      const bool runs = __all_sync(0xffffffffu, t.run > 0 && row >= 0 && row == run_first + in_run);
      uint32_t from[8], from_t[4];                         // this lane's rows of the copies, four and eight rows an instruction
#pragma unroll
      for (int k = 0; k < 8; ++k) from[k] = static_cast<uint32_t>(__shfl_sync(0xffffffffu, row, k * 4 + (lane >> 3)));
#pragma unroll
      for (int k = 0; k < 4; ++k) from_t[k] = static_cast<uint32_t>(__shfl_sync(0xffffffffu, row, k * 8 + (lane >> 2)));
      const int row0 = __shfl_sync(0xffffffffu, row, 0), row16 = __shfl_sync(0xffffffffu, row, 16);
      for (int c = 0; c <= pl.n_full && ok; ++c) {         // c = n_full: the tail
        if (c == pl.n_full && !pl.tail) break;
        const bool is_tail = c == pl.n_full;
        const int slot = s * pl.n_full + c, col = (c < n_kf || is_tail ? (is_tail ? n_kf : c) : c + gap) * 128;
        uint64_t* full_bar = is_tail ? &tfull[ts] : &full[slot];
        ok = __all_sync(0xffffffffu, is_tail ? mbar_wait(&tempty[ts], tph ^ 1, abort_flag) : mbar_wait(&empty[slot], ph ^ 1, abort_flag));
        if (!ok) break;
        const uint32_t width = is_tail ? 64 : 128;
        uint8_t* const to = (is_tail ? tails + ts * kTailBytes : ring + static_cast<size_t>(slot) * kChunkBytes) + warp * 32 * width;
        if (runs) {
          if (lane == 0) {
            expect_bytes(full_bar, 32 * width);
            if (is_tail) {
              tma_load_3d(to, &map_tail, col, head, row0, full_bar, policy);
              if (t.run == 16) tma_load_3d(to + 16 * 64, &map_tail, col, head, row16, full_bar, policy);
            } else {
              tma_load_3d(to, &map, col, head, row0, full_bar, policy);
              if (t.run == 16) tma_load_3d(to + 16 * 128, &map, col, head, row16, full_bar, policy);
            }
          }
          __syncwarp();
          mbar_arrive(full_bar);
        } else if (!is_tail) {
          const int piece = lane & 7, r_in = lane >> 3;
          const bool in = col + piece * 16 < g.W;          // past the row's end there is nothing to read
          const uint8_t* base = g.rows + static_cast<size_t>(head) * g.W + (in ? col + piece * 16 : 0);
          const uint32_t at = smem_u32(to) + r_in * 128;
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const bool real = static_cast<int>(from[k]) >= 0;
            copy16(at + k * 512 + ((piece ^ (((k & 1) << 2) + r_in)) * 16), base + (real ? from[k] * row_bytes : 0), real && in ? 16u : 0u);
          }
          copies_arrive(full_bar);
        } else {
          const int piece = lane & 3, r_in = lane >> 2;
          const bool in = col + piece * 16 < g.W;
          const uint8_t* base = g.rows + static_cast<size_t>(head) * g.W + (in ? col + piece * 16 : 0);
          const uint32_t at = smem_u32(to) + r_in * 64 + ((piece ^ ((r_in >> 1) & 3)) * 16);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const bool real = static_cast<int>(from_t[k]) >= 0;
            copy16(at + k * 512, base + (real ? from_t[k] * row_bytes : 0), real && in ? 16u : 0u);
          }
          copies_arrive(full_bar);
        }
      }
      if (!ok) break;
      // every slot was free, so the weights of the stage's last tile have been read
      info[s * kTile + threadIdx.x] = make_float2(scale, __int_as_float(word));
      mbar_arrive(&ifull[s]);
      if (++s == pl.stages) { s = 0; ph ^= 1; }
      if (++ts == pl.tstages) { ts = 0; tph ^= 1; }
      tok1 = tok2; main1 = main2; page1 = page2; scale1 = scale2;
      tok2 = tok3; main2 = main3;
    }
    // every copy has landed before the block goes on: on the way out of an abort too
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (!ok) drain_boxes();
  } else if (warp == kMmaWarp) {
    // ---------------------------------------------------------------- MMA issuer
    if (lane == 0) {
      const uint32_t ring_u = smem_u32(ring), q_u = smem_u32(qimg), p_u = smem_u32(pbuf), tail_u = smem_u32(tails);
      const int n_kf = pl.n_k - pl.tail, n_f = pl.n_full, n_v = pl.n_v;
      const int v_slot0 = plan_v_slot(pl, pl.v0);          // value chunks lie in consecutive slots from here
      constexpr uint32_t id_s = idesc(2 * C, 0, 0), id_hi = idesc(C, 0, 1), id_lo = idesc(C, 1, 1);
      const uint64_t ring_d = desc128(ring_u), q_d = desc128(q_u), p_d = desc128(p_u), tail_d = desc64(tail_u),
                     qt_d = desc64(q_u + n_kf * (2 * C * 128));
      bool ok = n == 0 || mbar_wait(qfull, 0, abort_flag);
      // Steps of one chunk, whichever is ready: the scores of tile js (at most one tile ahead of
      // the values, for two S buffers), or the values of tile jv once its weights are there.
      int js = 0, cs = 0, ss = 0, tss = 0, jv = 0, cv = 0, sv = 0;   // tile, chunk, stage (and tail)
      uint32_t ph = 0, tph = 0, phv = 0;
      const int s_steps = n_kf + pl.tail;
      uint32_t idle = 0;
      unsigned long long t0 = 0;
      while (ok && jv < n) {
        bool moved = false;
        if (js < n && js <= jv + 1) {
          const uint32_t d_t = tmem + (js & 1) * (2 * C);
          const uint32_t acc = cs > 0 ? 1u : 0u;
          if (cs < n_kf) {
            const int slot = ss * n_f + cs;
            if (mbar_try_wait(&full[slot], ph)) {
              asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // the copies, to the MMAs
              tc_fence_after();
              const uint64_t ad = ring_d + slot * (kChunkBytes >> 4), bd = q_d + cs * ((2 * C * 128) >> 4);
              const int left = pl.ksteps - 4 * cs;
              mma<true>(d_t, ad, bd, id_s, acc);
              if (left > 1) mma<true>(d_t, ad + 2, bd + 2, id_s, 1u);
              if (left > 2) mma<true>(d_t, ad + 4, bd + 4, id_s, 1u);
              if (left > 3) mma<true>(d_t, ad + 6, bd + 6, id_s, 1u);
              if (cs < v_slot0 || cs >= v_slot0 + n_v) mma_commit(&empty[slot]);   // keys alone
              moved = true;
            }
          } else if (mbar_try_wait(&tfull[tss], tph)) {
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            tc_fence_after();
            mma<true>(d_t, tail_d + tss * (kTailBytes >> 4), qt_d, id_s, acc);
            if (pl.ksteps - 4 * n_kf > 1) mma<true>(d_t, tail_d + tss * (kTailBytes >> 4) + 2, qt_d + 2, id_s, 1u);
            mma_commit(&tempty[tss]);
            if (++tss == pl.tstages) { tss = 0; tph ^= 1; }
            moved = true;
          }
          if (moved && ++cs == s_steps) {
            mma_commit(&sfull[js & 1]);
            ++js;
            cs = 0;
            if (++ss == pl.stages) { ss = 0; ph ^= 1; }
          }
        }
        if (!moved && jv < js) {
          const int c = v_slot0 + cv, slot = sv * n_f + c;
          if ((cv > 0 || mbar_try_wait(pfull, jv & 1)) && (c < n_kf || mbar_try_wait(&full[slot], phv))) {
            if (c >= n_kf) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            tc_fence_after();
            const uint64_t ad = ring_d + slot * (kChunkBytes >> 4);
            const uint32_t d_t = tmem + kO + cv * C;
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) {
              mma<true>(d_t, ad + ks * 256, p_d + ks * 256, id_hi, jv > 0 || ks > 0 ? 1u : 0u);
              mma<true>(d_t, ad + ks * 256, p_d + ks * 256 + 4, id_lo, 1u);
            }
            mma_commit(&empty[slot]);
            moved = true;
            if (++cv == n_v) {
              mma_commit(pdone);
              cv = 0;
              ++jv;
              if (++sv == pl.stages) { sv = 0; phv ^= 1; }
            }
          }
        }
        if (moved) {
          idle = 0;
        } else if ((++idle & 63u) == 0) {                  // bounded like every wait
          if (idle == 64) t0 = global_timer();
          if (*abort_flag || global_timer() - t0 > kWaitLimitNs) {
            *abort_flag = 1;
            ok = false;
          }
        }
      }
      mma_commit(drain);
      volatile int no_abort = 0;
      mbar_wait(drain, 0, &no_abort);
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------------- weights and results
    const int wg = (warp - 4) >> 2, quad = warp & 3, row = quad * 32 + lane;
    const int c0 = wg * NC, bar_id = 1 + wg;               // wg: group of four warps, one per TMEM lane quadrant
    const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
    // The query image: row c the first terms of column c, row C + c the second ones.  The
    // rows of missing columns and the elements past d are zeros.
    {
      constexpr int kBatch = 4;                            // columns a warp loads at a time
      const int n_kf = pl.n_k - pl.tail, dpad = pl.ksteps * 32;
      const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q);
#pragma unroll 1
      for (int cb = 0; cb < C / Sh::kWeights; cb += kBatch) {
        uint4 v[kBatch][3];                                // d <= 576: at most 72 groups of 8
#pragma unroll
        for (int k2 = 0; k2 < kBatch; ++k2) {
          const int c = (cb + k2) * Sh::kWeights + warp - 4, col = c_base + c, i = col / hg;
          const __nv_bfloat16* qrow = q + ((static_cast<size_t>(b) * a.Tq + i) * a.H + head * hg + (col - i * hg)) * a.d;
#pragma unroll
          for (int k = 0; k < 3; ++k) {
            const int e = (lane + 32 * k) * 8;
            v[k2][k] = c < n_c && e < a.d ? __ldg(reinterpret_cast<const uint4*>(qrow + e)) : make_uint4(0, 0, 0, 0);
          }
        }
#pragma unroll
        for (int k2 = 0; k2 < kBatch; ++k2) {
          const int c = (cb + k2) * Sh::kWeights + warp - 4;
          uint32_t m = 0;
#pragma unroll
          for (int k = 0; k < 3; ++k) {
            const uint32_t w[4] = {v[k2][k].x, v[k2][k].y, v[k2][k].z, v[k2][k].w};
#pragma unroll
            for (int x = 0; x < 4; ++x) m = max(m, max((w[x] << 16) & 0x7fffffffu, w[x] & 0x7fff0000u));
          }
          m = __reduce_max_sync(0xffffffffu, m);
          const bool finite = m < 0x7f800000u;
          // s = 2^e, the smallest (from 2^-100) with max|q| / s <= 448
          const int se = max(static_cast<int>(m >> 23) - 8 + ((m & 0x7fffffu) > 0x600000u ? 1 : 0), 27);
          const float inv = finite ? __uint_as_float(static_cast<uint32_t>(254 - se) << 23) : 0.f;
          if (lane == 0) {
            const float sc = finite ? __uint_as_float(static_cast<uint32_t>(se) << 23) : __uint_as_float(0x7fc00000u);
            qf[c] = c < n_c ? sc * a.sm * 1.44269504088896f : 0.f;
            nref[c] = kUnset;
            qi[c] = static_cast<uint16_t>(min(c_base + c, ncol - 1) / hg);
          }
#pragma unroll
          for (int k = 0; k < 3; ++k) {
            const int e = (lane + 32 * k) * 8;
            if (e >= dpad) continue;
            const uint32_t w[4] = {v[k2][k].x, v[k2][k].y, v[k2][k].z, v[k2][k].w};
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
            const int chunk = e / 128, j = (e % 128) / 16, x = e % 16;   // C is a multiple of 8: one swizzle for both rows
            const bool main_chunk = chunk < n_kf;
            uint8_t* base = qimg + (main_chunk ? chunk : n_kf) * (2 * C * 128) +
                            (main_chunk ? c * 128 + ((j ^ (c & 7)) * 16) : c * 64 + ((j ^ ((c >> 1) & 3)) * 16)) + x;
            *reinterpret_cast<uint2*>(base) = hv;
            *reinterpret_cast<uint2*>(base + C * (main_chunk ? 128 : 64)) = lv;
          }
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(qfull);
      asm volatile("barrier.cta.sync 3, %0;" ::"n"(32 * Sh::kWeights) : "memory");   // the columns' factors, to all
    }
    // Scratch of 256 words for the group, in its own columns' bytes of the weights buffer (two
    // words a row), while no MMA reads them.
    auto scratch = [&](int i) {
      const int r = i >> 1;
      return reinterpret_cast<float*>(pbuf + r * 128 + (((c0 >> 4) ^ (r & 7)) * 16) + (c0 & 15) + (i & 1) * 4);
    };
    float2 l[NC / 2];
#pragma unroll
    for (int c = 0; c < NC / 2; ++c) l[c] = make_float2(0.f, 0.f);
    const float target = fminf(fmaxf(lg2(static_cast<float>(max(n, 1))) - 1.f, 0.f), 6.f);   // log2(128 n) - 8
    bool ok = true;
    int s = 0;
    uint32_t ph = 0;
#pragma unroll 1
    for (int j = 0; j < n; ++j) {
      if (ok) ok = mbar_wait(&ifull[s], ph, abort_flag);
      const float2 in = info[s * kTile + row];
      const float scale = in.x;
      const int word = __float_as_int(in.y);
      // an unseen token has scale 0: its exponent is 0 + log2(0) = -infinity
      const float ls = scale == 0.f ? -INFINITY : lg2(scale);
      uint32_t seen = 0xffffffffu;                         // columns of this group that see the token
      if (a.Tq > 1 && !__all_sync(0xffffffffu, word < 0 || scale == 0.f)) {
        if (word >= 0) {
          seen = 0;
#pragma unroll 1
          for (int c = 0; c < NC; ++c) {
            const bool in_main = kv_sees(a, word & (kListFlag - 1), sp.len - a.Tq + qi[c0 + c]);
            seen |= (in_main != ((word & kListFlag) != 0) ? 1u : 0u) << c;
          }
        }
      }
      if (ok) ok = mbar_wait(&sfull[j & 1], (j >> 1) & 1, abort_flag);
      tc_fence_after();
      // Exponents above the reference (pass 0 and 2) or as they are (pass 1: the reference is set
      // anew, for the first tile and when a weight passes its limit).
      float y[NC];
      bool stop = false;
#pragma unroll 1
      for (int pass = j == 0 ? 1 : 0; pass < 3; ++pass) {
        const float2 with_ref = pass == 1 ? make_float2(0.f, 0.f) : make_float2(1.f, 1.f);
        uint32_t hi[NC], lo[NC];
        const uint32_t st = tmem + lanes + (j & 1) * (2 * C) + c0;
        tmem_ld(st, hi);
        tmem_ld(st + C, lo);
        tmem_wait_ld();
        const float2 ls2 = make_float2(ls, ls), sc2 = make_float2(scale, scale);
#pragma unroll
        for (int c = 0; c < NC; c += 4) {
          const float4 f = *reinterpret_cast<const float4*>(qf + c0 + c), r = *reinterpret_cast<const float4*>(nref + c0 + c);
          const float2 x0 = mul2(add2(pair(hi[c], hi[c + 1]), pair(lo[c], lo[c + 1])), sc2);
          const float2 x1 = mul2(add2(pair(hi[c + 2], hi[c + 3]), pair(lo[c + 2], lo[c + 3])), sc2);
          const float2 y0 = fma2(x0, make_float2(f.x, f.y), fma2(make_float2(r.x, r.y), with_ref, ls2));
          const float2 y1 = fma2(x1, make_float2(f.z, f.w), fma2(make_float2(r.z, r.w), with_ref, ls2));
          y[c] = y0.x;
          y[c + 1] = y0.y;
          y[c + 2] = y1.x;
          y[c + 3] = y1.y;
        }
        if (seen != 0xffffffffu) {
#pragma unroll
          for (int c = 0; c < NC; ++c)
            if (!((seen >> c) & 1)) y[c] = -INFINITY;
        }
        if (pass == 2) break;
        if (pass == 0) {
          float top = y[0];
#pragma unroll
          for (int c = 1; c < NC; ++c) top = fmaxf(top, y[c]);
          if (!group_any(bar_id, !ok || top > kLimit)) break;
          continue;
        }
        stop = group_any(bar_id, !ok);                     // the same for the whole group
        if (stop) break;
        // The weights buffer is scratch once the MMAs that read it are done.
        if (j > 0) ok = mbar_wait(pdone, (j - 1) & 1, abort_flag);
        tc_fence_after();
        float mine = -INFINITY;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          const float m = warp_max(y[c]);
          if (lane == c) mine = m;
        }
        if (lane < NC) *scratch(quad * 32 + lane) = mine;
        group_sync(bar_id);
        float f_mine = 1.f, now = 0.f;
        if (lane < NC) {
          const float old = nref[c0 + lane];
          const float m = fmaxf(fmaxf(*scratch(lane), *scratch(32 + lane)), fmaxf(*scratch(64 + lane), *scratch(96 + lane)));
          now = m + old > kLimit ? target - m : old;
          f_mine = now == old ? 1.f : ex2(now - old);      // 0 from unset
        }
        group_sync(bar_id);                                // every warp has read the old reference
        if (quad == 0 && lane < NC) nref[c0 + lane] = now;
#pragma unroll
        for (int c = 0; c < NC; ++c) (c & 1 ? l[c / 2].y : l[c / 2].x) *= __shfl_sync(0xffffffffu, f_mine, c);
        if (j > 0) {
#pragma unroll 1
          for (int m = 0; m < pl.n_v; ++m) {
            const uint32_t at = tmem + lanes + kO + m * C + c0;
            tmem_ld(at, hi);
            tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < NC; ++c) hi[c] = __float_as_uint(__uint_as_float(hi[c]) * __shfl_sync(0xffffffffu, f_mine, c));
            tmem_st(at, hi);
          }
          tmem_wait_st();
        }
        group_sync(bar_id);                                // the new reference, to all
      }
      if (stop) break;
      // Of a NaN scale only the columns that see the token become NaN.
      const float inv = scale > 0.f ? 1.0f / scale : 1.0f;
      uint32_t hw[NC / 4], lw[NC / 4];
#pragma unroll
      for (int c = 0; c < NC; c += 4) {
        const float2 p0 = make_float2(ex2(y[c]), ex2(y[c + 1])), p1 = make_float2(ex2(y[c + 2]), ex2(y[c + 3]));
        const float2 inv2 = make_float2(inv, inv);
        l[c / 2] = fma2(p0, inv2, l[c / 2]);
        l[c / 2 + 1] = fma2(p1, inv2, l[c / 2 + 1]);
        uint32_t h0, h1, l0, l1;
        split2(p0, h0, l0);
        split2(p1, h1, l1);
        hw[c / 4] = h0 | (h1 << 16);
        lw[c / 4] = l0 | (l1 << 16);
      }
      if (ok && j > 0) ok = mbar_wait(pdone, (j - 1) & 1, abort_flag);
      uint8_t* pr = pbuf + row * 128;
#pragma unroll
      for (int k = 0; k < NC / 16; ++k) {
        const int ch = c0 / 16 + k, cl = 4 + ch;
        *reinterpret_cast<uint4*>(pr + ((ch ^ (row & 7)) * 16)) = make_uint4(hw[4 * k], hw[4 * k + 1], hw[4 * k + 2], hw[4 * k + 3]);
        *reinterpret_cast<uint4*>(pr + ((cl ^ (row & 7)) * 16)) = make_uint4(lw[4 * k], lw[4 * k + 1], lw[4 * k + 2], lw[4 * k + 3]);
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(pfull);
      if (++s == pl.stages) { s = 0; ph ^= 1; }
    }
    // The last tile's values are in.  Sums over the block's tokens, and O^T into the ring as
    // [C][128 n_v] fp32 (every tile has been read).
    if (ok && n > 0) ok = mbar_wait(pdone, (n - 1) & 1, abort_flag);
    tc_fence_after();
    float mine = 0.f;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      float v = c & 1 ? l[c / 2].y : l[c / 2].x;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      if (lane == c) mine = v;
    }
    if (lane < NC) *scratch(quad * 32 + lane) = mine;
    group_sync(bar_id);
    if (quad == 0 && lane < NC)
      qf[c0 + lane] = (*scratch(lane) + *scratch(32 + lane)) + (*scratch(64 + lane) + *scratch(96 + lane));
    float* os = reinterpret_cast<float*>(ring) + row;
    const int pitch = pl.n_v * 128;
#pragma unroll 1
    for (int m = 0; m < pl.n_v; ++m) {
      uint32_t o[NC];
#pragma unroll
      for (int c = 0; c < NC; ++c) o[c] = 0u;
      if (n > 0) {
        tmem_ld(tmem + lanes + kO + m * C + c0, o);
        tmem_wait_ld();
      }
      float* to = os + m * 128 + c0 * pitch;
#pragma unroll
      for (int c = 0; c < NC; ++c) to[c * pitch] = __uint_as_float(o[c]);
    }
  }
  tc_fence_before();
  if (t.cluster > 1) cluster_sync();
  else __syncthreads();
  if (threadIdx.x == 0 && *abort_flag) raise_status(a.status, LSA_ERR_TIMEOUT);
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
  // ------------------------------------------------------------------ join
  // This block's share of the columns: out = sum_x w_x O_x, w_x = 2^(r_x - r) (over the sum of
  // the weights when the unit has one cluster).
  {
    const int X = t.cluster, share = C / X, cs = rank * share;
    float* wtab = reinterpret_cast<float*>(pbuf);          // [X][share]: weights
    float2* rl = reinterpret_cast<float2*>(pbuf + C * 4);  // [X][share]: reference, sum
    if (threadIdx.x < C) {
      const int x = threadIdx.x / share, c = cs + threadIdx.x - x * share;
      rl[threadIdx.x] = make_float2(-peer_ld(peer(smem_u32(nref + c), x)), peer_ld(peer(smem_u32(qf + c), x)));
    }
    __syncthreads();
    if (threadIdx.x < share) {
      const int c = cs + threadIdx.x, col = c_base + c;
      float m = -kUnset, sum = 0.f;
      for (int x = 0; x < X; ++x) {
        const float2 v = rl[x * share + threadIdx.x];
        if (v.y != 0.f) m = fmaxf(m, v.x);
      }
      for (int x = 0; x < X; ++x) {
        const float2 v = rl[x * share + threadIdx.x];
        if (v.y != 0.f) sum = fmaf(ex2(v.x - m), v.y, sum);
      }
      const float r = a.splits > 1 ? 1.f : sum == 0.f ? 0.f : 1.0f / sum;
      for (int x = 0; x < X; ++x) {
        const float2 v = rl[x * share + threadIdx.x];
        wtab[x * share + threadIdx.x] = v.y != 0.f ? ex2(v.x - m) * r : 0.f;
      }
      if (c < n_c) {
        if (a.splits == 1) {
          const size_t oc = (static_cast<size_t>(b) * a.Tq + col / hg) * a.H + head * hg + col % hg;
          if (a.lse) a.lse[oc] = sum == 0.f ? -INFINITY : (m + log2f(sum)) * 0.693147180559945f;
        } else {
          const size_t pc = ((static_cast<size_t>(b) * g.G + head) * a.splits + grp) * ncol + col;
          a.part_m[pc] = m;
          a.part_l[pc] = sum;
        }
      }
    }
    __syncthreads();
    const int pitch = pl.n_v * 128, shift = a.voff - pl.v0 * 128;
    const bool vec = a.dv % 4 == 0 && shift % 4 == 0;
    const uint32_t base = smem_u32(ring);
    const int mine = max(0, min(share, n_c - cs));
    // A warp takes a column's values 128 at a time (four a lane); one value a lane where the
    // value columns do not start or end on a multiple of four.
    const int step = vec ? 128 : 32, per = (a.dv + step - 1) / step;
    auto join_columns = [&](auto count) {
      constexpr int kX = decltype(count)::value;
#pragma unroll 2
      for (int i = warp; i < mine * per; i += kThreads / 32) {
        const int cl = i / per, v = (i - cl * per) * step + lane * (vec ? 4 : 1);
        if (v >= a.dv) continue;
        const uint32_t at = base + static_cast<uint32_t>(((cs + cl) * pitch + shift + v) * 4);
        float o[4] = {0.f, 0.f, 0.f, 0.f};
        if (vec) {
          float4 f[kX];
#pragma unroll
          for (int x = 0; x < kX; ++x) f[x] = peer_ld4(peer(at, x));
#pragma unroll
          for (int x = 0; x < kX; ++x) {
            const float w = wtab[x * share + cl];
            o[0] = fmaf(w, f[x].x, o[0]);
            o[1] = fmaf(w, f[x].y, o[1]);
            o[2] = fmaf(w, f[x].z, o[2]);
            o[3] = fmaf(w, f[x].w, o[3]);
          }
        } else {
          for (int x = 0; x < kX; ++x) o[0] = fmaf(wtab[x * share + cl], peer_ld(peer(at, x)), o[0]);
        }
        const int col = c_base + cs + cl;
        if (a.splits == 1) {
          const size_t oc = (static_cast<size_t>(b) * a.Tq + col / hg) * a.H + head * hg + col % hg;
          __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + oc * a.dv + v;
          if (vec) {
            const __nv_bfloat162 p0 = __floats2bfloat162_rn(o[0], o[1]), p1 = __floats2bfloat162_rn(o[2], o[3]);
            *reinterpret_cast<uint2*>(out) = make_uint2(*reinterpret_cast<const uint32_t*>(&p0), *reinterpret_cast<const uint32_t*>(&p1));
          } else {
            out[0] = __float2bfloat16_rn(o[0]);
          }
        } else {
          const size_t pc = ((static_cast<size_t>(b) * g.G + head) * a.splits + grp) * ncol + col;
          if (vec) *reinterpret_cast<float4*>(a.part_o + pc * a.dv + v) = make_float4(o[0], o[1], o[2], o[3]);
          else a.part_o[pc * a.dv + v] = o[0];
        }
      }
    };
    switch (X) {
      case 1: join_columns(std::integral_constant<int, 1>{}); break;
      case 2: join_columns(std::integral_constant<int, 2>{}); break;
      case 4: join_columns(std::integral_constant<int, 4>{}); break;
      default: join_columns(std::integral_constant<int, 8>{}); break;
    }
  }
  if (t.cluster > 1) cluster_sync();                       // nobody reads this block's shared memory any more
}

int columns(int ncol) { return ncol <= 16 ? 16 : ncol <= 32 ? 32 : 64; }

// Two blocks share an SM where each gets two stages of its half; one block has it all otherwise.
Plan plan_for(int d, int dv, int voff, int C) {
  if (C < 64) {
    const Plan half = make_plan(d, dv, voff, C, kSmemLimit / 2 - 1024);
    if (half.stages >= 2) return half;
  }
  return make_plan(d, dv, voff, C, kSmemLimit);
}

template <int C>
int launch_c(const CUtensorMap& map, const CUtensorMap& tail, const AttendTc& t, long long grid, cudaStream_t s) {
  const cudaError_t e = cudaFuncSetAttribute(kv_attend_tc_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, t.p.smem);
  if (e != cudaSuccess) return fail(LSA_ERR_CUDA, "kv_attend: %s", cudaGetErrorString(e));
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = t.cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(Shape<C>::kThreads);
  cfg.dynamicSmemBytes = t.p.smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaLaunchKernelEx(&cfg, kv_attend_tc_kernel<C>, map, tail, t);
  return check_launch("kv_attend");
}

}  // namespace

bool kv_attend_tc_supported(long long max_tokens, int d, int dv, int voff, int qdt, int ncol) {
  // 16384 tokens a part, at most 8 parts a cluster and 256 clusters a unit; tokens below 2^30
  if (qdt != LSA_BF16 || d % 8 != 0 || d > 576 || max_tokens > 16384ll * 8 * 256) return false;
  const Plan p = plan_for(d, dv, voff, columns(ncol));
  return p.n_v <= 4 && p.stages >= 2 && p.smem <= kSmemLimit;
}

void kv_attend_parts_tc(int B, int G, int ncol, long long max_tokens, int& cluster, int& groups) {
  const int C = columns(ncol);
  const long long units = static_cast<long long>(B) * G * ((ncol + C - 1) / C);
  const long long tiles = std::max<long long>(1, (max_tokens + kTile - 1) / kTile);
  const long long least = (max_tokens + 16383) / 16384;   // parts, by the weights' range (see the top)
  // A division costs its waves of blocks times a block's tiles, its start and end counted as three
  // tiles (two blocks of an SM take its time in turn, so they count as two waves); a second kernel that joins clusters as three and their sums' traffic.  Clusters of 4
  // and 8 leave some SMs of a graphics cluster unused.
  const int xs[4] = {1, 2, 4, 8}, slots[4] = {148, 148, 144, 128};
  long long best = -1;
  for (int k = 0; k < 4; ++k) {
    const long long X = xs[k], room = slots[k];
    if (X > 1 && X > tiles) break;
    for (long long gr = std::max<long long>(1, (least + X - 1) / X); gr <= 256; ++gr) {
      if (best >= 0 && X * gr > tiles) break;
      const long long waves = (units * gr * X + room - 1) / room;
      const long long c = 16 * waves * ((tiles + X * gr - 1) / (X * gr) + 3) + (gr > 1 ? 48 + gr : 0) + 4 * k;
      if (best < 0 || c < best) {
        best = c;
        cluster = static_cast<int>(X);
        groups = static_cast<int>(gr);
      }
      if (units * gr * X > 16 * 148) break;
    }
  }
}

int launch_kv_attend_tc(const KvAttendArgs& a, int cluster, cudaStream_t s) {
  const int ncol = a.Tq * (a.H / a.g.G), C = columns(ncol);
  AttendTc t{};
  t.a = a;
  t.p = plan_for(a.d, a.dv, a.voff, C);
  t.col_groups = (ncol + C - 1) / C;
  t.cluster = cluster;
  const long long grid = static_cast<long long>(a.g.B) * a.g.G * a.splits * t.col_groups * cluster;
  // Rows of consecutive tokens follow one another within a page (a whole sequence without a table).
  CUtensorMap map{}, tail{};
  const KvGeom& g = a.g;
  const long long rows = static_cast<long long>(g.pages) << g.page_log;
  t.run = rows < 32 ? 0 : g.table == nullptr || g.page_log >= 5 ? 32 : g.page_log == 4 ? 16 : 0;
  if (t.run > 0) {
    EncodeTiledFn enc = encode_fn();
    if (!enc) return fail(LSA_ERR_CUDA, "kv_attend: cuTensorMapEncodeTiled unavailable");
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(g.W), static_cast<cuuint64_t>(g.G), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(g.W), static_cast<cuuint64_t>(g.G) * g.W};
    const cuuint32_t estr[3] = {1, 1, 1};
    const cuuint32_t box[3] = {128, 1, static_cast<cuuint32_t>(t.run)}, box_tail[3] = {64, 1, static_cast<cuuint32_t>(t.run)};
    CUresult cr = enc(&map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, g.rows, dims, strides, box, estr,
                      CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (cr == CUDA_SUCCESS)
      cr = enc(&tail, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, g.rows, dims, strides, box_tail, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (cr != CUDA_SUCCESS) return fail(LSA_ERR_CUDA, "kv_attend: tensor map encode failed (%d)", static_cast<int>(cr));
  }
  if (C == 64) return launch_c<64>(map, tail, t, grid, s);
  if (C == 32) return launch_c<32>(map, tail, t, grid, s);
  return launch_c<16>(map, tail, t, grid, s);
}

}  // namespace lsa
