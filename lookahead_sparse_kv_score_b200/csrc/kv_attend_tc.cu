// Attention over the 8-bit KV cache on the tensor cores of sm_100a: TMA boxes or copies of rows ->
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
// Rounding.  A bf16 query element has 8 significant bits; scaled by a power of two to at most 448,
// an e4m3 term holds the first four and a second one the rest, exactly, except below 2^-10 / 224 of
// the row's largest element.  A weight P'' (see below) is rounded to fp16 and held as an e4m3 and
// an e5m2 term, in units that put the largest at 2^6 to 2^12.  From 2^-6 of a unit on, half a step
// of both terms is at most 2^-8 of the weight, which is what a bf16 weight is off by (rms 1.2e-3, a
// bf16 weight 1.6e-3): a second term in e5m2 leaves that much behind one in e4m3, and one in e4m3
// behind e5m2, which is how weights above 448 are held.  Below, half a step is 2^-14 of a unit, an
// eighth of the weight or 2^-17 of a unit, whichever is less at its size: so weights keep bf16's
// precision down to 2^-12 of the largest before them.  A heavy token that carries little value must
// not cost the others theirs: the unit moves back behind it (see below), and in its own tile the
// largest is put at 2^12, so that the precision reaches down to 2^-18 of it (2^-12 where heavy
// tokens stand among each of the four warps' shares of a tile).  Parts have at most 16384 tokens,
// so that the weights lost below 2^-17 of a unit are less than 2^-9 of the sum.  Scores, the sum of
// the weights and the accumulators are fp32.
//
// Scales.  y_tc = sm log2(e) scale_t (q_c . k_t) + log2 |scale_t|; the value weight is P''_tc =
// 2^(y_tc - r_c) with the scale's sign and the softmax weight P''_tc / |scale_t|, so one
// exponential serves both sums and the scale never multiplies the codes.  r_c is set so that the
// largest weight seen is 2^6 and kept until a weight would pass 2^12: then the block's O^T columns
// are multiplied by 2^(r_old - r_new) in tensor memory.  (A part of one tile, and a tile in which
// one warp's tokens all weigh far less than the largest, take 2^12 at once.)  It moves back, by up
// to 40 bits, when the tile behind a move stays below 2^-2; that tile alone is looked at, as a
// first token of large weight, or a later one, is what makes it so.  Moves are rare after the first
// tile, so the cross-lane maxima are only computed then; otherwise a tile costs one vote.  The room
// of six bits is what uneven scales need: with 2^8 as the target the drafted window takes 37 us
// instead of 32.
//
// Roles (10, 14 or 22 warps by the columns).  Warps 0-3 bring the rows, one token a lane, chunk
// by chunk, and write the tokens' scales.  Four warps for each 16 columns make the weights, one
// token a lane.  The last two issue the MMAs of S and of O, a chunk at a time as chunks arrive and
// weights are ready, S a tile ahead of O.  Rows that follow one another in memory (a dense
// cache, pages of 16 and more) come as TMA boxes; other rows (a fetched list) by 16-byte
// asynchronous copies in the MMA's swizzle, with zeros where a place has no token: with 64 KB
// in flight an SM, random 128-byte pieces come at 19 bytes a clock by copies and at 13 by TMA row
// gathers.
//
// What bounds it.  With few query columns, memory: 16384 tokens x 8 KV heads x 256 bytes, B = 32,
// read at 5.6 TB/s (146.8 us).  With 64 columns on latent rows a tile's products take 1.4 us at shared memory's
// rate (an MMA of N = 128 takes 64 clocks, of N = 64 48: its operands' bytes), and the chain of a
// tile (rows 0.9 us, S 0.6 to 1.5, weights 1.4, O 0.8 to 1.4) over the two tiles that fit beside
// the query image comes to 2.5 to 2.8 us, against 1.7 for its bytes.  The join of a cluster is bound by
// distributed shared memory (14 to 16 bytes a clock and SM however it is moved): 5 us for 64
// columns of 512 values in four blocks, which is why short calls take fewer columns a block.
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
#include <cmath>
#include <type_traits>

#include "kv_common.cuh"
#include "tc_ptx.cuh"

namespace lsa {
namespace {

using namespace tc;

constexpr int kTile = 128;
constexpr int kProducers = 128;               // warps 0-3

// A block's shape by its query columns: a group of four weights warps (one a quadrant of the
// tensor memory's lanes) for each 16 columns; up to 32 columns, two blocks share an SM.
constexpr int NC = 16;                        // columns of a weights warp
template <int C>
struct Shape {
  static constexpr int kWeights = 4 * (C / NC);            // warps
  static constexpr int kMmaWarp = 4 + kWeights;            // the first of two: scores, values
  static constexpr int kThreads = 32 * (kMmaWarp + 2);
  static constexpr int kBlocks = C == 64 ? 1 : 2;          // blocks an SM, where shared memory allows
  static constexpr uint32_t kTmemCols = C == 64 ? 512 : C == 32 ? 256 : 128;
};
constexpr int kSmemLimit = 227 * 1024;
constexpr int kChunkBytes = kTile * 128;      // 128 columns of a tile, 128-byte swizzle
constexpr int kTailBytes = kTile * 64;        // the last 64 key columns, 64-byte swizzle
constexpr int kMaxStages = 4;
constexpr int kMaxSlots = 12;                 // stages times 128-column chunks: 16 KB each
constexpr int kBars = 46;                     // 8-byte words of barriers and flags
constexpr int kMaxCluster = 8;
constexpr float kUnset = 3.0e38f;             // minus the reference exponent before any token was seen
constexpr float kLimit = 12.f;                // exponents of weights: reference kept up to here
constexpr float kTarget = 6.f;                // the largest weight's when the reference is set
constexpr float kApart = 8.f;                 // bits between two warps' largest weights that are far apart
constexpr float kLow = -2.f;                  // the largest weight's of a tile, below which the reference may move back
constexpr float kBack = 40.f;                 // bits that it moves back at most
constexpr float kTiny = 0x1p-60f;             // smaller scales count as 0
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
  const int p_bytes = 2 * kTile * C;                           // weights, first and second terms
  const int fixed = q_bytes + p_bytes + kBars * 8 + C * (8 + 2);
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
  p.t_off = p.p_off + p_bytes;
  p.i_off = p.t_off + p.tail * p.tstages * kTailBytes;
  p.m_off = p.i_off + p.stages * kTile * 8;
  p.smem = p.m_off + kBars * 8 + C * (8 + 2);
  return p;
}

struct AttendTc {
  KvAttendArgs a;
  Plan p;
  int col_groups, cluster, hg;
  int run;          // rows of a TMA box (16 or 32 places whose rows follow one another), 0: no maps
};

// Shared-memory matrix descriptors: start address and version word; groups of eight rows (a
// row is 128 or 64 bytes, as wide as the swizzle) `group` bytes apart; swizzle 2 (128 bytes) or 4 (64).
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr) { return ((saddr >> 4) & 0x3FFFu) | (1u << 16); }
__host__ __device__ constexpr uint32_t desc_hi(uint32_t group, uint32_t swizzle) {
  return (group >> 4) | (1u << 14) | (swizzle << 29);
}
// The weights are not swizzled: blocks of 16 columns, [128 tokens][16 bytes] each.  Eight tokens
// (128 bytes) are a core matrix; the leading offset goes to the next eight, the stride to the
// next 16 columns.
__device__ __forceinline__ uint32_t desc_p_lo(uint32_t saddr) { return ((saddr >> 4) & 0x3FFFu) | ((128u >> 4) << 16); }

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
__device__ __forceinline__ void tmem_ld(uint32_t t, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];" : LSA_R8(r, 0) : "r"(t));
}
__device__ __forceinline__ void tmem_ld(uint32_t t, uint32_t& r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r) : "r"(t));
}
__device__ __forceinline__ void tmem_st(uint32_t t, uint32_t r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%1], {%0};" ::"r"(r), "r"(t) : "memory");
}
__device__ __forceinline__ void tmem_st(uint32_t t, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::LSA_I8(r, 0), "r"(t) : "memory");
}
__device__ __forceinline__ void tmem_st(uint32_t t, const uint32_t (&r)[16]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, "
               "%13, %14, %15};" ::LSA_I8(r, 0), LSA_I8(r, 8), "r"(t) : "memory");
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
// log2 of a positive normal number: the exponent apart, so that a power of two's is exact (the weights are
// divided by the scale itself: an error here would stay in them).
__device__ __forceinline__ float log2_of(float x) {
  const int e = static_cast<int>(__float_as_uint(x) - 0x3f800000u) >> 23;
  return static_cast<float>(e) + lg2(__uint_as_float(__float_as_uint(x) - (static_cast<uint32_t>(e) << 23)));
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

// The MMA warps run converged and an elected lane issues.  A descriptor's low word is made
// uniform once a chunk, so that the ones behind it are sums in uniform registers: an MMA then
// takes its 48 clocks (N = 64; 64 with N = 128, shared memory's rate), where descriptors in
// vector registers made it 97.
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); }
__device__ __forceinline__ bool elect() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(r)::"memory");
  return r != 0;
}
__device__ __forceinline__ void mma_lo(uint32_t d_tmem, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo, uint32_t b_hi, uint32_t id,
                                       uint32_t acc) {
  asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tmov.b64 a, {%1, %2};\n\tmov.b64 b, {%3, %4};\n\tsetp.ne.b32 p, %6, 0;\n\t"
               "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %5, p;\n\t}" ::"r"(d_tmem), "r"(a_lo), "r"(a_hi),
               "r"(b_lo), "r"(b_hi), "r"(id), "r"(acc) : "memory");
}

// Adds to the bytes a barrier's phase waits for, without arriving.
__device__ __forceinline__ void expect_bytes(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void prefetch(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }
// L2 policy of the rows' boxes: rows that one block reads leave first (16384 tokens x 8 KV heads, B = 32:
// 2% less time), rows that several blocks of a unit read do not.
__device__ __forceinline__ uint64_t rows_policy(bool once) {
  uint64_t p;
  if (once) asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  else asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
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
// The weights warps' sums, to the producers of a block without a cluster: kWait for those that wait.
template <int kCount, bool kWait>
__device__ __forceinline__ void stats_barrier() {
  if constexpr (kWait) asm volatile("barrier.cta.sync 7, %0;" ::"n"(kCount) : "memory");
  else asm volatile("barrier.cta.arrive 7, %0;" ::"n"(kCount) : "memory");
}
// All threads of the cluster, each warp converged: writes before the arrival are seen by reads behind the wait.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_sync() {
  cluster_arrive();
  cluster_wait();
}

// Two weights (at most 2^12) as e4m3 codes (hi) and e5m2 codes (lo) of the two terms that they are held
// as.  Up to 448 the e4m3 term comes first and the other takes what is left; above, the e5m2 term
// does: fp16's sign, exponent and first two fraction bits, rounded by adding half of the last
// (the carry stays in its half: the values are far below fp16's largest), and at most 256 are left.
__device__ __forceinline__ void split2(float2 p, uint32_t& hi, uint32_t& lo) {
  const __half2 w = __floats2half2_rn(p.x, p.y);
  const uint32_t above = __hgt2_mask(w, __floats2half2_rn(448.f, 448.f));
  const uint32_t first = (*reinterpret_cast<const uint32_t*>(&w) + 0x00800080u) & 0xff00ff00u & above;
  const __half2 w1 = __hsub2(w, *reinterpret_cast<const __half2*>(&first));
  const __nv_fp8x2_storage_t h = __nv_cvt_halfraw2_to_fp8x2(__half2_raw(w1), __NV_SATFINITE, __NV_E4M3);
  const __half2 rest = __hsub2(w1, __half2(__nv_cvt_fp8x2_to_halfraw2(h, __NV_E4M3)));
  const uint32_t second = (*reinterpret_cast<const uint32_t*>(&rest) & ~above) | first;
  hi = h;
  lo = __nv_cvt_halfraw2_to_fp8x2(__half2_raw(*reinterpret_cast<const __half2*>(&second)), __NV_SATFINITE, __NV_E5M2);
}

__device__ __forceinline__ void store_words(uint8_t* p, const uint32_t (&w)[4]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store_words(uint8_t* p, const uint32_t (&w)[2]) { *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]); }

// Blocks of a unit: rank (fastest), column group, cluster of the unit's parts, KV head, sequence.
template <int C>
__global__ void __launch_bounds__(Shape<C>::kThreads, Shape<C>::kBlocks)
kv_attend_tc_kernel(const __grid_constant__ CUtensorMap map, const __grid_constant__ CUtensorMap map_tail,
                    const __grid_constant__ AttendTc t) {
  using Sh = Shape<C>;
  constexpr int kMmaWarp = Sh::kMmaWarp, kThreads = Sh::kThreads;
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
  uint64_t* drain = bars + 41;              // both MMA warps
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 42);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + 43);
  uint64_t* sempty = bars + 44;             // [2]

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int hg = t.hg, ncol = a.Tq * hg;
  // (a division only where there is something to divide)
  uint32_t u = blockIdx.x;
  auto digit = [&](int count) -> int {
    if (count == 1) return 0;
    const uint32_t q = u / count, r = u - q * count;
    u = q;
    return static_cast<int>(r);
  };
  const int rank = digit(t.cluster), cg = digit(t.col_groups), grp = digit(a.splits), head = digit(g.G);   // a.splits: clusters of a unit
  const int b = static_cast<int>(u);
  const int c_base = cg * C, n_c = min(C, ncol - c_base);
  const int parts = a.splits * t.cluster, part = grp * t.cluster + rank;

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
    mbar_init(drain, 2);
    mbar_init(&sempty[0], Sh::kWeights);
    mbar_init(&sempty[1], Sh::kWeights);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  // The kernel before may still run: what it may write is only fetched to L2 here (this part's list
  // entries, the lengths, the query rows), and read behind the wait.
  if (warp < 4) {
    if (a.idx != nullptr) {
      const long long e1 = static_cast<long long>(a.cap) * (part + 1) / parts;
      for (long long e = static_cast<long long>(a.cap) * part / parts + threadIdx.x * 32; e < e1; e += kProducers * 32)
        prefetch(a.idx + static_cast<size_t>(b) * a.cap + e);
      if (threadIdx.x == 1) prefetch(a.count + b);
    }
    if (threadIdx.x == 0) prefetch(a.length + b);
  }
  if (warp >= 4 && warp < kMmaWarp) {
    const int c = (warp - 4) * 4 + (lane >> 3), col = c_base + c, i = a.Tq == 1 ? 0 : col / hg;   // eight lanes a row
    if (c < n_c) {
      const char* qrow = reinterpret_cast<const char*>(static_cast<const __nv_bfloat16*>(a.q) +
                                                       ((static_cast<size_t>(b) * a.Tq + i) * a.H + head * hg + (col - i * hg)) * a.d);
      for (int e = (lane & 7) * 128; e < a.d * 2; e += 1024) prefetch(qrow + e);
    }
  }
  // What follows reads the call's inputs, by plain loads, and allocates tensor memory (which the kernel
  // before may not have done yet).
  pdl_wait();
  if (warp == kMmaWarp) tmem_alloc(tmem_slot, kTmemCols);
  const KvSpan sp = kv_span(a, b);
  const int tiles = (sp.total + kTile - 1) / kTile;
  const int each = parts == 1 ? tiles : tiles / parts, more = tiles - each * parts;   // the first `more` parts have one tile more
  const int tile0 = part * each + min(part, more), n = each + (part < more ? 1 : 0);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // The cluster's first meeting: every block's references and sums are set.  Only the weights warps
  // have something to bring to it, and only the producers wait for it before their work is done.
  const bool met = t.cluster > 1;
  if (met && (warp < 4 || warp >= kMmaWarp)) cluster_arrive();

  if (warp < 4) {
    // ---------------------------------------------------------------- producers
    const int p_first = sp.len - a.Tq + (c_base / hg), p_last = sp.len - a.Tq + (c_base + n_c - 1) / hg;
    const int n_kf = pl.n_k - pl.tail, gap = max(pl.v0 - n_kf, 0);   // chunks between keys and values are not read
    const size_t row_bytes = static_cast<size_t>(g.G) * g.W;
    const uint64_t policy = rows_policy(t.col_groups == 1);
    const int v_slot0 = plan_v_slot(pl, pl.v0), v_last = v_slot0 + pl.n_v - 1;
    // A value slot whose release says that every chunk of the stage's last tile has arrived: the scores
    // have waited for the chunks with keys before the first values begin; chunks without keys are
    // waited for one by one, so then it is the last.
    const int v_done = v_last >= n_kf ? v_last : v_slot0;
    const bool divide = t.run > 0 && pl.n_full >= 3;
    const int piece = lane & 7, r_in = lane >> 3;          // a lane's 16 bytes of a chunk and its row of four
    const uint8_t* lane_base = g.rows + static_cast<size_t>(head) * g.W + piece * 16;
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
      page = g.table != nullptr ? g.table[static_cast<size_t>(b) * g.n_pages + (tok >> g.page_log)] : tok >> g.page_log;
      sc = g.scale[kv_scale_at(g, b, tok, head)];
    };
    // The token's row (-1: nothing to read), scale (0: nobody sees it) and word.  A stored scale of 0 is a
    // row of zeros at the smallest scale: its score is 0 and it counts among the weights.
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
      if (fabsf(sc) < kTiny) {
        row = -1;
        scale = kTiny;
      }
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
      // A warp brings its 32 rows, chunk by chunk: boxes where they are runs, else copies.  Tiles of
      // three and more chunks whose rows are all runs are divided by chunks instead, so that a slot
      // is filled as soon as it is free whatever the others wait for (two barriers a tile: not
      // worth it for one or two chunks, 175 against 161 us on 16384 tokens x 8 KV heads, B = 32).
      float2* words = info + s * kTile;
      bool by_chunks = false;
      if (divide) {
        // The stage's token words are free once the values of its last tile have begun; they carry
        // the runs' first rows to the warps.
        if (ok) ok = mbar_wait(&empty[s * pl.n_full + v_done], ph ^ 1, abort_flag);
        words[threadIdx.x].x = __int_as_float(row);
        by_chunks = !group_any(6, !runs || !ok);
      }
      if (by_chunks) {
        // The others' chunks get nothing from this warp (their slots' last phase is over, by the wait
        // for v_done).
        for (int c = 0; c < pl.n_full; ++c)
          if ((c & 3) != warp) mbar_arrive(&full[s * pl.n_full + c]);
        for (int c = warp; c < pl.n_full + pl.tail; c += 4) {
          const bool is_tail = c == pl.n_full;
          const int slot = s * pl.n_full + c, col = (is_tail ? n_kf : c < n_kf ? c : c + gap) * 128;
          uint64_t* full_bar = is_tail ? &tfull[ts] : &full[slot];
          if (!__all_sync(0xffffffffu, mbar_wait(is_tail ? &tempty[ts] : &empty[slot], (is_tail ? tph : ph) ^ 1, abort_flag))) {
            ok = false;
            break;
          }
          if (lane == 0) expect_bytes(full_bar, is_tail ? kTailBytes : kChunkBytes);
          __syncwarp();
          mbar_arrive(full_bar);
          if (lane < kTile / t.run) {                      // a lane a box
            const int r = lane * t.run, row0 = __float_as_int(words[r].x);
            if (is_tail) tma_load_3d(tails + ts * kTailBytes + r * 64, &map_tail, col, head, row0, full_bar, policy);
            else tma_load_3d(ring + static_cast<size_t>(slot) * kChunkBytes + r * 128, &map, col, head, row0, full_bar, policy);
          }
        }
        __syncwarp();
        if (pl.tail && (pl.n_full & 3) != warp) {          // one tail may serve all stages: its last phase must be over
          if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&tempty[ts], tph ^ 1, abort_flag));
          if (ok) mbar_arrive(&tfull[ts]);
        }
        if (group_any(6, !ok)) break;                      // (and every warp has read the rows)
      } else {
        if (divide && group_any(6, !ok)) break;            // the same for the four warps
        const int row0 = __shfl_sync(0xffffffffu, row, 0), row16 = __shfl_sync(0xffffffffu, row, 16);
        const uint8_t* src[8];                             // this lane's rows of the copies, four rows an instruction
        uint32_t there = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int r = __shfl_sync(0xffffffffu, row, k * 4 + r_in);
          there |= (r >= 0 ? 1u : 0u) << k;
          src[k] = lane_base + static_cast<size_t>(max(r, 0)) * row_bytes;
        }
        // the tail before the last chunk: its slot is free earlier
        for (int step = 0; step < pl.n_full + pl.tail; ++step) {
          const bool is_tail = pl.tail && step == pl.n_full - 1;
          const int c = pl.tail && step == pl.n_full ? step - 1 : step;
          const int slot = s * pl.n_full + c, col = (is_tail ? n_kf : c < n_kf ? c : c + gap) * 128;
          if (ok) ok = __all_sync(0xffffffffu, mbar_wait(is_tail ? &tempty[ts] : &empty[slot], (is_tail ? tph : ph) ^ 1, abort_flag));
          if (!ok) continue;
          if (runs) {
            uint64_t* full_bar = is_tail ? &tfull[ts] : &full[slot];
            if (lane == 0) {
              if (is_tail) {
                uint8_t* to = tails + ts * kTailBytes + warp * 2048;
                expect_bytes(full_bar, 2048);
                tma_load_3d(to, &map_tail, col, head, row0, full_bar, policy);
                if (t.run == 16) tma_load_3d(to + 1024, &map_tail, col, head, row16, full_bar, policy);
              } else {
                uint8_t* to = ring + static_cast<size_t>(slot) * kChunkBytes + warp * 4096;
                expect_bytes(full_bar, 4096);
                tma_load_3d(to, &map, col, head, row0, full_bar, policy);
                if (t.run == 16) tma_load_3d(to + 2048, &map, col, head, row16, full_bar, policy);
              }
            }
            __syncwarp();
            mbar_arrive(full_bar);
          } else if (!is_tail) {
            const bool in = col + piece * 16 < g.W;        // past the row's end there is nothing to read
            const uint32_t at0 = smem_u32(ring) + slot * kChunkBytes + warp * 4096 + r_in * 128 + ((piece ^ r_in) * 16), at1 = at0 ^ 64;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const bool real = in && ((there >> k) & 1);
              copy16(((k & 1) ? at1 : at0) + k * 512, src[k] + (in ? col : 0), real ? 16u : 0u);
            }
            copies_arrive(&full[slot]);
          } else {
            const int p4 = lane & 3, r8 = lane >> 2;       // eight rows an instruction
            const bool in = col + p4 * 16 < g.W;
            const uint8_t* base = g.rows + static_cast<size_t>(head) * g.W + (in ? col + p4 * 16 : 0);
            const uint32_t at = smem_u32(tails) + ts * kTailBytes + warp * 2048 + r8 * 64 + ((p4 ^ ((r8 >> 1) & 3)) * 16);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int r = __shfl_sync(0xffffffffu, row, k * 8 + r8);
              copy16(at + k * 512, base + static_cast<size_t>(max(r, 0)) * row_bytes, r >= 0 && in ? 16u : 0u);
            }
            copies_arrive(&tfull[ts]);
          }
        }
      }
      if (!divide && !ok) break;
      words[threadIdx.x] = make_float2(scale, __int_as_float(word));
      mbar_arrive(&ifull[s]);
      if (++s == pl.stages) { s = 0; ph ^= 1; }
      if (++ts == pl.tstages) { ts = 0; tph ^= 1; }
      tok1 = tok2; main1 = main2; page1 = page2; scale1 = scale2;
      tok2 = tok3; main2 = main3;
    }
    // every copy has landed before the block goes on: on the way out of an abort too
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (*abort_flag) drain_boxes();
  } else if (warp >= kMmaWarp) {
    // ---------------------------------------------------------------- MMA issuers
    // One warp for the scores and one for the values: an issue waits while the tensor core is
    // busy, and a barrier test or a commit (100 to 150 clocks) in between would leave it idle.
    const int n_kf = pl.n_k - pl.tail, n_f = pl.n_full, n_v = pl.n_v, n_sc = n_kf + pl.tail;
    const int v_slot0 = plan_v_slot(pl, pl.v0);            // value chunks lie in consecutive slots from here
    constexpr uint32_t id_s = idesc(2 * C, 0, 0), id_hi = idesc(C, 0, 1), id_lo = idesc(C, 1, 1);
    constexpr uint32_t kHi128 = desc_hi(1024, 2), kHi64 = desc_hi(512, 4);
    const uint32_t ring_lo = desc_lo(smem_u32(ring));
    auto wait = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag)); };
    bool ok = true;
    if (warp == kMmaWarp) {
      const uint32_t q_lo = desc_lo(smem_u32(qimg)), tail_lo = desc_lo(smem_u32(tails)), qt_lo = desc_lo(smem_u32(qimg) + n_kf * (2 * C * 128));
      int s = 0, ts = 0;
      uint32_t ph = 0, tph = 0;
      if (n > 0) ok = wait(qfull, 0);
      for (int j = 0; ok && j < n; ++j) {
        ok = wait(&sempty[j & 1], ((j >> 1) & 1) ^ 1);
        const uint32_t d_t = uniform(tmem + (j & 1) * (2 * C));
        for (int c = 0; ok && c < n_kf; ++c) {
          const int slot = s * n_f + c;
          if (!(ok = wait(&full[slot], ph))) break;
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // the copies, to the MMAs
          tc_fence_after();
          const int left = pl.ksteps - 4 * c;
          const uint32_t ad = uniform(ring_lo + slot * (kChunkBytes >> 4)), bd = uniform(q_lo + c * ((2 * C * 128) >> 4));
          if (elect()) {
            mma_lo(d_t, ad, kHi128, bd, kHi128, id_s, c > 0 ? 1u : 0u);
            if (left > 1) mma_lo(d_t, ad + 2, kHi128, bd + 2, kHi128, id_s, 1u);
            if (left > 2) mma_lo(d_t, ad + 4, kHi128, bd + 4, kHi128, id_s, 1u);
            if (left > 3) mma_lo(d_t, ad + 6, kHi128, bd + 6, kHi128, id_s, 1u);
            if (c < v_slot0 || c >= v_slot0 + n_v) mma_commit(&empty[slot]);   // keys alone
            if (c + 1 == n_sc) mma_commit(&sfull[j & 1]);
          }
          __syncwarp();
        }
        if (ok && pl.tail && (ok = wait(&tfull[ts], tph))) {
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          tc_fence_after();
          const uint32_t ad = uniform(tail_lo + ts * (kTailBytes >> 4)), bd = uniform(qt_lo);
          if (elect()) {
            mma_lo(d_t, ad, kHi64, bd, kHi64, id_s, n_kf > 0 ? 1u : 0u);
            if (pl.ksteps - 4 * n_kf > 1) mma_lo(d_t, ad + 2, kHi64, bd + 2, kHi64, id_s, 1u);
            mma_commit(&sfull[j & 1]);
            mma_commit(&tempty[ts]);
          }
          __syncwarp();
        }
        if (++s == pl.stages) { s = 0; ph ^= 1; }
        if (++ts == pl.tstages) { ts = 0; tph ^= 1; }
      }
    } else {
      const uint32_t bd = uniform(desc_p_lo(smem_u32(pbuf)));
      constexpr uint32_t kHiP = desc_hi(2048, 0);
      int s = 0;
      uint32_t ph = 0;
      for (int j = 0; ok && j < n; ++j) {
        if (!(ok = wait(pfull, j & 1))) break;
        const uint32_t acc = j > 0 ? 1u : 0u;
        for (int m = 0; m < n_v; ++m) {
          const int c = v_slot0 + m, slot = s * n_f + c;
          if (c >= n_kf) {                                 // a chunk without keys: nobody has waited for it yet
            if (!(ok = wait(&full[slot], ph))) break;
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          }
          tc_fence_after();
          const uint32_t ad = uniform(ring_lo + slot * (kChunkBytes >> 4)), d_t = uniform(tmem + kO + m * C);
          if (elect()) {
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) {
              mma_lo(d_t, ad + ks * 256, kHi128, bd + ks * 32, kHiP, id_hi, ks > 0 ? 1u : acc);
              mma_lo(d_t, ad + ks * 256, kHi128, bd + ks * 32 + (C / 16) * 128, kHiP, id_lo, 1u);
            }
            mma_commit(&empty[slot]);
            if (m + 1 == n_v) mma_commit(pdone);
          }
          __syncwarp();
        }
        if (++s == pl.stages) { s = 0; ph ^= 1; }
      }
    }
    // every MMA this warp issued is done before the tensor memory is given up (commits count the
    // elected lane's: it issued them all)
    if (elect()) {
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
          const int c = (cb + k2) * Sh::kWeights + warp - 4, col = c_base + c, i = a.Tq == 1 ? 0 : col / hg;
          const __nv_bfloat16* qrow = q + ((static_cast<size_t>(b) * a.Tq + i) * a.H + head * hg + (col - i * hg)) * a.d;
#pragma unroll
          for (int k = 0; k < 3; ++k) {
            const int e = (lane + 32 * k) * 8;
            v[k2][k] = c < n_c && e < a.d ? *reinterpret_cast<const uint4*>(qrow + e) : make_uint4(0, 0, 0, 0);
          }
        }
        float inv[kBatch];
#pragma unroll
        for (int k2 = 0; k2 < kBatch; ++k2) {
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
          inv[k2] = finite ? __uint_as_float(static_cast<uint32_t>(254 - se) << 23) : 0.f;
          if (lane == 0) {
            const int c = (cb + k2) * Sh::kWeights + warp - 4;
            const float sc = finite ? __uint_as_float(static_cast<uint32_t>(se) << 23) : __uint_as_float(0x7fc00000u);
            qf[c] = c < n_c ? sc * a.sm * 1.44269504088896f : 0.f;
            nref[c] = kUnset;
            qi[c] = static_cast<uint16_t>(a.Tq == 1 ? 0 : min(c_base + c, ncol - 1) / hg);
          }
        }
#pragma unroll
        for (int k = 0; k < 3; ++k) {
          const int e = (lane + 32 * k) * 8;
          if (e >= dpad) continue;
          const int chunk = e >> 7, j = (e & 127) >> 4;
          const bool main_chunk = chunk < n_kf;
          uint8_t* at = qimg + (main_chunk ? chunk : n_kf) * (2 * C * 128) + (e & 8);
          const int second = C * (main_chunk ? 128 : 64);  // C is a multiple of 8: one swizzle for both rows
#pragma unroll
          for (int k2 = 0; k2 < kBatch; ++k2) {
            const int c = (cb + k2) * Sh::kWeights + warp - 4;
            const uint32_t w[4] = {v[k2][k].x, v[k2][k].y, v[k2][k].z, v[k2][k].w};
            const float2 inv2 = make_float2(inv[k2], inv[k2]);
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const float2 f = mul2(pair(w[x] << 16, w[x] & 0xffff0000u), inv2);
              hi[x] = __nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3);
              const float2 h = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(hi[x]), __NV_E4M3)));
              lo[x] = __nv_cvt_float2_to_fp8x2(make_float2(f.x - h.x, f.y - h.y), __NV_SATFINITE, __NV_E4M3);
            }
            uint8_t* base = at + (main_chunk ? c * 128 + ((j ^ (c & 7)) * 16) : c * 64 + ((j ^ ((c >> 1) & 3)) * 16));
            *reinterpret_cast<uint2*>(base) = make_uint2(hi[0] | (hi[1] << 16), hi[2] | (hi[3] << 16));
            *reinterpret_cast<uint2*>(base + second) = make_uint2(lo[0] | (lo[1] << 16), lo[2] | (lo[3] << 16));
          }
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(qfull);
      asm volatile("barrier.cta.sync 5, %0;" ::"n"(32 * Sh::kWeights) : "memory");   // the columns' factors, to all
    }
    // NA: 16 (NC), or 8 where the block has no more columns (what lies behind is not read): 16384 tokens x 8 KV
    // heads of 8 columns, B = 32, take 147 us, 154 with 16.  One group of several on its own code is
    // slower (20 columns, 4096 tokens x 7 heads, B = 8: by 2.5 us).
    auto weigh = [&](auto active) {
      constexpr int NA = decltype(active)::value;
      // Scratch of 512 words for the group, in its own columns' block of the weights buffer, while no
      // MMA reads it.
      auto scratch = [&](int i) { return reinterpret_cast<float*>(pbuf + wg * 2048) + i; };
      float2 l[NA / 2];
#pragma unroll
      for (int c = 0; c < NA / 2; ++c) l[c] = make_float2(0.f, 0.f);
      bool ok = true, fresh = false;                         // fresh: a reference was set or moved in the tile before
      float lowest = kUnset;                                 // of column `lane`: the smallest nref so far
      int s = 0;
      uint32_t ph = 0;
#pragma unroll 1
      for (int j = 0; j < n; ++j) {
        if (ok) ok = mbar_wait(&ifull[s], ph, abort_flag);
        const float2 in = info[s * kTile + row];
        const float scale = in.x;
        const int word = __float_as_int(in.y);
        // an unseen token has scale 0: its exponent is 0 + log2(0) = -infinity
        const float ls = scale == 0.f ? -INFINITY : log2_of(fabsf(scale));
        uint32_t seen = 0xffffffffu;                         // columns of this group that see the token
        if (a.Tq > 1 && !__all_sync(0xffffffffu, word < 0 || scale == 0.f)) {
          if (word >= 0) {
            seen = 0;
#pragma unroll 1
            for (int c = 0; c < NA; ++c) {
              const bool in_main = kv_sees(a, word & (kListFlag - 1), sp.len - a.Tq + qi[c0 + c]);
              seen |= (in_main != ((word & kListFlag) != 0) ? 1u : 0u) << c;
            }
          }
        }
        if (ok) ok = mbar_wait(&sfull[j & 1], (j >> 1) & 1, abort_flag);
        tc_fence_after();
        // Exponents above the reference (pass 0 and 2) or as they are (pass 1: the reference is set
        // anew, for the first tile and when a weight passes its limit).
        float y[NA];
        bool stop = false;
#pragma unroll 1
        for (int pass = j == 0 ? 1 : 0; pass < 3; ++pass) {
          const float2 with_ref = pass == 1 ? make_float2(0.f, 0.f) : make_float2(1.f, 1.f);
          uint32_t hi[NA], lo[NA];
          const uint32_t st = tmem + lanes + (j & 1) * (2 * C) + c0;
          tmem_ld(st, hi);
          tmem_ld(st + C, lo);
          tmem_wait_ld();
          const float2 ls2 = make_float2(ls, ls), sc2 = make_float2(scale, scale);
#pragma unroll
          for (int c = 0; c < NA; c += 4) {
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
            for (int c = 0; c < NA; ++c)
              if (!((seen >> c) & 1)) y[c] = -INFINITY;
          }
          if (pass == 2) break;
          if (pass == 0) {
            float top = y[0];
#pragma unroll
            for (int c = 1; c < NA; ++c) top = fmaxf(top, y[c]);
            if (group_any(bar_id, !ok || top > kLimit)) continue;
            if (!fresh) break;
            // Whether in each warp (that has tokens) all weights of some column are small.
            fresh = false;
            uint32_t high = 0;
#pragma unroll
            for (int c = 0; c < NA; ++c) high |= (y[c] > kLow ? 1u : 0u) << c;
            high = __reduce_or_sync(0xffffffffu, high);
            if (group_any(bar_id, high == (1u << NA) - 1 && __any_sync(0xffffffffu, scale != 0.f))) break;
            continue;
          }
          stop = group_any(bar_id, !ok);                     // the same for the whole group
          if (stop) break;
          // The weights buffer is scratch once the MMAs that read it are done.
          if (j > 0) ok = mbar_wait(pdone, (j - 1) & 1, abort_flag);
          tc_fence_after();
          float mine = -INFINITY;
#pragma unroll
          for (int c = 0; c < NA; ++c) {
            const float m = warp_max(y[c]);
            if (lane == c) mine = m;
          }
          if (lane < NA) *scratch(quad * 32 + lane) = mine;
          group_sync(bar_id);
          float f_mine = 1.f, now = 0.f;
          if (lane < NA) {
            const float old = nref[c0 + lane];
            const float m0 = *scratch(lane), m1 = *scratch(32 + lane), m2 = *scratch(64 + lane), m3 = *scratch(96 + lane);
            const float m01 = fmaxf(m0, m1), m23 = fmaxf(m2, m3), m = fmaxf(m01, m23);
            // No headroom where nothing comes behind, or where the weights of some warp are all far smaller (most
            // likely those of the next tile are too, and then the reference moves back).
            auto seen_or = [&](float x) { return x > -INFINITY ? x : m; };
            const float least = fminf(fminf(seen_or(m0), seen_or(m1)), fminf(seen_or(m2), seen_or(m3)));
            const float to = (n == 1 || m - least > kApart ? kLimit : kTarget) - m;
            now = m + old > kLimit ? to : m + old < kLow && m > -INFINITY ? fmaxf(old, fminf(to, lowest + kBack)) : old;
            lowest = fminf(lowest, now);
            f_mine = now == old ? 1.f : ex2(now - old);      // 0 from unset
          }
          group_sync(bar_id);                                // every warp has read the old reference
          if (quad == 0 && lane < NA) nref[c0 + lane] = now;
#pragma unroll
          for (int c = 0; c < NA; ++c) (c & 1 ? l[c / 2].y : l[c / 2].x) *= __shfl_sync(0xffffffffu, f_mine, c);
          const uint32_t moved = __ballot_sync(0xffffffffu, f_mine != 1.f);   // columns whose reference moved
          fresh = moved != 0;
          if (j > 0) {
#pragma unroll 1
            for (int m = 0; m < pl.n_v; ++m) {
              const uint32_t at = tmem + lanes + kO + m * C + c0;
              if (__popc(moved) > 4) {
                tmem_ld(at, hi);
                tmem_wait_ld();
#pragma unroll
                for (int c = 0; c < NA; ++c) hi[c] = __float_as_uint(__uint_as_float(hi[c]) * __shfl_sync(0xffffffffu, f_mine, c));
                tmem_st(at, hi);
              } else {
                for (uint32_t left = moved; left != 0; left &= left - 1) {
                  const int c = __ffs(left) - 1;
                  uint32_t o;
                  tmem_ld(at + c, o);
                  tmem_wait_ld();
                  tmem_st(at + c, __float_as_uint(__uint_as_float(o) * __shfl_sync(0xffffffffu, f_mine, c)));
                }
              }
            }
            tmem_wait_st();
          }
          group_sync(bar_id);                                // the new reference, to all
        }
        if (stop) break;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sempty[j & 1]);
        // Of a NaN scale only the columns that see the token become NaN.  A negative scale changes the codes' signs.
        const float inv = fabsf(scale) > 0.f ? 1.0f / fabsf(scale) : 1.0f;
        const uint32_t sign = scale < 0.f ? 0x80808080u : 0u;
        uint32_t hw[NA / 4], lw[NA / 4];
#pragma unroll
        for (int c = 0; c < NA; c += 4) {
          const float2 p0 = make_float2(ex2(y[c]), ex2(y[c + 1])), p1 = make_float2(ex2(y[c + 2]), ex2(y[c + 3]));
          const float2 inv2 = make_float2(inv, inv);
          l[c / 2] = fma2(p0, inv2, l[c / 2]);
          l[c / 2 + 1] = fma2(p1, inv2, l[c / 2 + 1]);
          uint32_t h0, h1, l0, l1;
          split2(p0, h0, l0);
          split2(p1, h1, l1);
          hw[c / 4] = (h0 | (h1 << 16)) ^ sign;
          lw[c / 4] = (l0 | (l1 << 16)) ^ sign;
        }
        if (ok && j > 0) ok = mbar_wait(pdone, (j - 1) & 1, abort_flag);
        uint8_t* pr = pbuf + wg * 2048 + row * 16;
        store_words(pr, hw);
        store_words(pr + (C / 16) * 2048, lw);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(pfull);
        if (++s == pl.stages) { s = 0; ph ^= 1; }
      }
      // Sums over the block's tokens, while the last tile's values are made, through the info of a stage
      // that every group has left.  Each step halves the columns a lane holds; lane l ends with
      // column l / (32 / NA).
      float v[NA];
#pragma unroll
      for (int c = 0; c < NA; ++c) v[c] = c & 1 ? l[c / 2].y : l[c / 2].x;
      int o = 16;
#pragma unroll
      for (int w = NA / 2; w >= 1; w /= 2) {
#pragma unroll
        for (int c = 0; c < w; ++c) {
          const bool up = (lane & o) != 0;
          const float keep = up ? v[c + w] : v[c], give = up ? v[c] : v[c + w];
          v[c] = keep + __shfl_xor_sync(0xffffffffu, give, o);
        }
        o >>= 1;
      }
      for (; o >= 1; o >>= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
      float* sums = reinterpret_cast<float*>(info + s * kTile) + wg * 64;      // [4][NA]
      sums[quad * NA + lane / (32 / NA)] = v[0];
      group_sync(bar_id);
      if (quad == 0 && lane < NA)
        qf[c0 + lane] = (sums[lane] + sums[NA + lane]) + (sums[2 * NA + lane] + sums[3 * NA + lane]);
      __syncwarp();
      if (met) cluster_arrive();
      else stats_barrier<32 * Sh::kWeights + kProducers, false>();
      // The last tile's values are in: O^T into the ring as [C][128 n_v] fp32 (every tile has been read).
      if (ok && n > 0) ok = mbar_wait(pdone, (n - 1) & 1, abort_flag);
      tc_fence_after();
      float* os = reinterpret_cast<float*>(ring) + row;
      const int pitch = pl.n_v * 128;
#pragma unroll 1
      for (int m = 0; m < pl.n_v; ++m) {
        uint32_t o[NA];
#pragma unroll
        for (int c = 0; c < NA; ++c) o[c] = 0u;
        if (n > 0) {
          tmem_ld(tmem + lanes + kO + m * C + c0, o);
          tmem_wait_ld();
        }
        float* to = os + m * 128 + c0 * pitch;
#pragma unroll
        for (int c = 0; c < NA; ++c) {
          *to = __uint_as_float(o[c]);
          to += pitch;
        }
      }
    };
    if (C == NC && n_c <= NC / 2) weigh(std::integral_constant<int, NC / 2>{});
    else weigh(std::integral_constant<int, NC>{});
  }
  // ------------------------------------------------------------------ join
  // This block's share of the columns: out = sum_x w_x O_x, w_x = 2^(r_x - r) (over the sum of
  // the weights when the unit has one cluster).  The producers make the w_x while the last values
  // are made and laid.
  const int X = t.cluster, share = C >> (31 - __clz(X)), cs = rank * share;
  float* wtab = reinterpret_cast<float*>(info);            // [X][share]: weights
  int* place = reinterpret_cast<int*>(info) + C;           // [share]: output row of a column
  __syncwarp();
  if (met) cluster_wait();
  else if (warp < 4) stats_barrier<32 * Sh::kWeights + kProducers, true>();
  if (static_cast<int>(threadIdx.x) < share) {             // at most the first two warps
    const int c = cs + static_cast<int>(threadIdx.x), col = c_base + c;
    float r[kMaxCluster], l[kMaxCluster], m = -kUnset, sum = 0.f;
#pragma unroll
    for (int x = 0; x < kMaxCluster; ++x) {
      r[x] = x < X ? -peer_ld(peer(smem_u32(nref + c), x)) : 0.f;
      l[x] = x < X ? peer_ld(peer(smem_u32(qf + c), x)) : 0.f;
    }
#pragma unroll
    for (int x = 0; x < kMaxCluster; ++x)
      if (l[x] != 0.f) m = fmaxf(m, r[x]);
#pragma unroll
    for (int x = 0; x < kMaxCluster; ++x) {
      r[x] = l[x] != 0.f ? ex2(r[x] - m) : 0.f;
      if (l[x] != 0.f) sum = fmaf(r[x], l[x], sum);
    }
    const float scale = a.splits > 1 ? 1.f : sum == 0.f ? 0.f : 1.0f / sum;
#pragma unroll
    for (int x = 0; x < kMaxCluster; ++x)
      if (x < X) wtab[x * share + threadIdx.x] = r[x] * scale;
    if (a.splits == 1) {
      const int i = a.Tq == 1 ? 0 : col / hg, oc = (b * a.Tq + i) * a.H + head * hg + col - i * hg;   // at most 2^24
      place[threadIdx.x] = oc;
      if (a.lse && c < n_c) a.lse[oc] = kv_lse(m, sum);
    } else {
      const size_t pc = ((static_cast<size_t>(b) * g.G + head) * a.splits + grp) * ncol + col;
      if (c < n_c) {
        a.part_m[pc] = m;
        a.part_l[pc] = sum;
      }
    }
  }
  __syncwarp();
  pdl_trigger();
  tc_fence_before();
  if (met) cluster_sync();                                 // sums and values of every block are laid
  else __syncthreads();
  if (threadIdx.x == 0 && *abort_flag) raise_status(a.status, LSA_ERR_TIMEOUT);
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
  {
    const int pitch = pl.n_v * 128, shift = a.voff - pl.v0 * 128;
    const bool vec = a.dv % 4 == 0 && shift % 4 == 0;
    const int mine = max(0, min(share, n_c - cs));
    float* part_o = a.part_o + ((((static_cast<size_t>(b) * g.G + head) * a.splits + grp) * ncol) + c_base + cs) * a.dv;
    __nv_bfloat16* outp = static_cast<__nv_bfloat16*>(a.out);
    if (vec) {
      // A warp keeps to 128 of a column's values (four a lane) and takes every few columns;
      // several columns' loads are in flight.
      const int per = (a.dv + 127) >> 7, lanes_of = (kThreads / 32) / per;   // 1 to 4 parts of a column
      const int p = warp / lanes_of, first = warp - p * lanes_of, v = p * 128 + lane * 4;
      auto join_columns = [&](auto count) {
        constexpr int kX = decltype(count)::value, kItems = kX >= 8 ? 1 : 8 / kX > 4 ? 4 : 8 / kX;   // eight loads in flight
        uint32_t from[kX];
#pragma unroll
        for (int x = 0; x < kX; ++x) from[x] = peer(smem_u32(ring) + static_cast<uint32_t>((cs * pitch + shift + v) * 4), x);
#pragma unroll 1
        for (int cl = first; cl < mine; cl += kItems * lanes_of) {
          float4 f[kItems][kX];
#pragma unroll
          for (int k = 0; k < kItems; ++k) {
            const uint32_t at = static_cast<uint32_t>(min(cl + k * lanes_of, mine - 1) * pitch * 4);
#pragma unroll
            for (int x = 0; x < kX; ++x) f[k][x] = peer_ld4(from[x] + at);
          }
#pragma unroll
          for (int k = 0; k < kItems; ++k) {
            const int c = cl + k * lanes_of;
            if (c >= mine) break;
            float2 o0 = make_float2(0.f, 0.f), o1 = o0;
#pragma unroll
            for (int x = 0; x < kX; ++x) {
              const float w = wtab[x * share + c];
              o0 = fma2(make_float2(w, w), make_float2(f[k][x].x, f[k][x].y), o0);
              o1 = fma2(make_float2(w, w), make_float2(f[k][x].z, f[k][x].w), o1);
            }
            if (a.splits == 1) {
              const __nv_bfloat162 p0 = __floats2bfloat162_rn(o0.x, o0.y), p1 = __floats2bfloat162_rn(o1.x, o1.y);
              *reinterpret_cast<uint2*>(outp + static_cast<size_t>(place[c]) * a.dv + v) =
                  make_uint2(*reinterpret_cast<const uint32_t*>(&p0), *reinterpret_cast<const uint32_t*>(&p1));
            } else {
              *reinterpret_cast<float4*>(part_o + static_cast<size_t>(c) * a.dv + v) = make_float4(o0.x, o0.y, o1.x, o1.y);
            }
          }
        }
      };
      if (p < per && v < a.dv) {
        switch (X) {
          case 1: join_columns(std::integral_constant<int, 1>{}); break;
          case 2: join_columns(std::integral_constant<int, 2>{}); break;
          case 4: join_columns(std::integral_constant<int, 4>{}); break;
          default: join_columns(std::integral_constant<int, 8>{}); break;
        }
      }
    } else {
      // value columns that do not start or end on a multiple of four: one a thread
      for (int i = threadIdx.x; i < mine * a.dv; i += kThreads) {
        const int c = i / a.dv, v = i - c * a.dv;
        const uint32_t at = smem_u32(ring) + static_cast<uint32_t>(((cs + c) * pitch + shift + v) * 4);
        float o = 0.f;
        for (int x = 0; x < X; ++x) o = fmaf(wtab[x * share + c], peer_ld(peer(at, x)), o);
        if (a.splits == 1) outp[static_cast<size_t>(place[c]) * a.dv + v] = __float2bfloat16_rn(o);
        else part_o[static_cast<size_t>(c) * a.dv + v] = o;
      }
    }
  }
  __syncwarp();
  if (met) cluster_sync();                                 // nobody reads this block's shared memory any more
}

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
  // the limit, not this call's size: two host threads may launch different sizes
  const cudaError_t e = cudaFuncSetAttribute(kv_attend_tc_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit);
  if (e != cudaSuccess) return fail(LSA_ERR_CUDA, "kv_attend: %s", cudaGetErrorString(e));
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = t.cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(Shape<C>::kThreads);
  cfg.dynamicSmemBytes = t.p.smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cudaLaunchKernelEx(&cfg, kv_attend_tc_kernel<C>, map, tail, t);
  return check_launch("kv_attend");
}

// Sizes of a cluster, and the blocks resident at once (the occupancy calculator's answers on B200:
// clusters of 4 and 8 leave some SMs of a graphics cluster unused), twice that with two blocks an SM.
constexpr int kSizes[4] = {1, 2, 4, 8}, kRoom[4] = {148, 148, 132, 120};

}  // namespace

int kv_attend_columns_tc(int B, int G, int ncol, long long max_tokens, int d, int dv, int voff, int qdt) {
  // 16384 tokens a part, at most 8 parts a cluster and 256 clusters a unit
  if (qdt != LSA_BF16 || d % 8 != 0 || d > 576 || max_tokens > 16384ll * 8 * 256) return 0;
  // The columns a block can hold; fewer where one wave of blocks takes them with four tiles a block or
  // less all the same: a quarter of the columns is a quarter of the query image to make and of the
  // sums to join (64 heads of latent rows: 512 rows, one sequence, 11 us with 16 columns a block, 19 with
  // 64; 300 rows, B = 16, 13.1 against 18.4; 1000 rows, B = 8, 14.1 against 18.6).
  const long long tiles = std::max<long long>(1, (max_tokens + kTile - 1) / kTile);
  auto one_wave = [&](long long units) {
    for (int k = 0; k < 4; ++k)
      if ((tiles + kSizes[k] - 1) / kSizes[k] <= 4 && units * kSizes[k] <= kRoom[k]) return true;
    return false;
  };
  for (int C = 16; C <= 64; C *= 2) {
    const bool enough = ncol <= C || C == 64;
    if (!enough && !one_wave(static_cast<long long>(B) * G * ((ncol + C - 1) / C))) continue;
    const Plan p = plan_for(d, dv, voff, C);
    if (p.n_v <= 4 && p.stages >= 2 && p.smem <= kSmemLimit) return C;
    if (enough) return 0;
  }
  return 0;
}

void kv_attend_parts_tc(int B, int G, int ncol, int C, int d, int dv, int voff, long long max_tokens, int& cluster, int& groups) {
  const long long units = static_cast<long long>(B) * G * ((ncol + C - 1) / C);
  const long long tiles = std::max<long long>(1, (max_tokens + kTile - 1) / kTile);
  const long long least = (max_tokens + 16383) / 16384;   // parts, by the weights' range (see the top)
  // A division costs the tiles of a block, its start and end counted as three, times: 1.5 for
  // a block alone on an SM that could hold two, 2 for two of them, more by the waves; a second
  // kernel that joins clusters as three tiles and their sums' traffic (131072 latent tokens: 47.4 us by
  // 74 clusters of two, 1.0 more by 33 of four; 20000 tokens of 256 codes, 128 columns: 21.2 and, by 16 of four,
  // 20.0).
  const Plan plan = plan_for(d, dv, voff, C);
  const double per_sm = C < 64 && plan.smem <= kSmemLimit / 2 - 1024 ? 2.0 : 1.0;
  const double traffic = plan.n_full >= 3 ? 40.0 : 16.0;   // a cluster's sums are a smaller part of a tile of wide rows
  double best = -1.0;
  for (int k = 0; k < 4; ++k) {
    const long long X = kSizes[k];
    if (X > 1 && X > tiles) break;
    for (long long gr = std::max<long long>(1, (least + X - 1) / X); gr <= 256; ++gr) {
      if (best >= 0.0 && X * gr > tiles) break;
      const double blocks = static_cast<double>(units * gr * X), room = kRoom[k] * per_sm;
      const double w = static_cast<double>((tiles + X * gr - 1) / (X * gr) + 3);
      double c = blocks <= kRoom[k] ? w * (per_sm > 1.0 ? 1.5 : 1.0)
                 : blocks <= room ? w * 2.2
                                  : per_sm * w * (per_sm > 1.0 ? blocks / room + 0.25 : std::ceil(blocks / room));
      c += (gr > 1 ? (3.0 + gr / traffic) * (per_sm > 1.0 ? 3.0 : 1.0) : 0.0) + 0.25 * k;
      if (best < 0.0 || c < best) {
        best = c;
        cluster = static_cast<int>(X);
        groups = static_cast<int>(gr);
      }
      if (blocks > 16 * 148) break;
    }
  }
}

int launch_kv_attend_tc(const KvAttendArgs& a, int C, int cluster, cudaStream_t s) {
  const int ncol = a.Tq * (a.H / a.g.G);
  AttendTc t{};
  t.a = a;
  t.p = plan_for(a.d, a.dv, a.voff, C);
  t.col_groups = (ncol + C - 1) / C;
  t.cluster = cluster;
  t.hg = a.H / a.g.G;
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
