// The 8-bit KV cache: rows quantised as they are written, and read back.
//
// A row is W e4m3 codes and belongs to one token and head; the rows of `block` consecutive
// tokens of a head share one fp32 scale s, the smallest power of two with amax / s <= 448
// (at least 2^-24, so that a block of zeros leaves a later token of the block its range).
// With a power of two the division is exact, so a code is its value rounded once, and a
// block whose scale grows when tokens are appended has its earlier codes divided by an
// exact power of two again.
//
// Both kernels move each byte once and are bound by memory.
#include <algorithm>
#include <type_traits>

#include "kv_common.cuh"

namespace lsa {
namespace {

constexpr int kThreads = 256;
constexpr int kFlight = 4;            // vectors a lane of the read has in flight
constexpr uint32_t kNanBits = 0x7fc00000u;

// Eight consecutive elements as they lie in memory.
struct Raw32 { uint4 a, b; };
struct Raw16 { uint4 a; };
__device__ __forceinline__ Raw32 load8(const float* p) {
  return {__ldg(reinterpret_cast<const uint4*>(p)), __ldg(reinterpret_cast<const uint4*>(p) + 1)};
}
__device__ __forceinline__ Raw16 load8(const __nv_bfloat16* p) { return {__ldg(reinterpret_cast<const uint4*>(p))}; }
__device__ __forceinline__ void to_floats(const Raw32& r, float (&v)[8]) {
  const uint32_t w[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
}
__device__ __forceinline__ void to_floats(const Raw16& r, float (&v)[8]) {
  const uint32_t w[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
// Largest magnitude as its bits: non-finite values have the largest of all.
__device__ __forceinline__ uint32_t amax_bits(const Raw32& r) {
  const uint32_t w[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, w[i] & 0x7fffffffu);
  return m;
}
__device__ __forceinline__ uint32_t amax_bits(const Raw16& r) {      // two 16-bit maxima an instruction
  const uint32_t k = 0x7fff7fffu;
  const uint32_t m = __vmaxu2(__vmaxu2(r.a.x & k, r.a.y & k), __vmaxu2(r.a.z & k, r.a.w & k));
  return max(m << 16, m & 0xffff0000u);
}

__device__ __forceinline__ uint2 encode8(const float (&v)[8], float inv) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = __nv_cvt_float2_to_fp8x2(make_float2(v[2 * i] * inv, v[2 * i + 1] * inv), __NV_SATFINITE, __NV_E4M3);
  return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

__device__ __forceinline__ void decode2(uint32_t w, float s, float& a, float& b) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w), __NV_E4M3);
  const float2 f = __half22float2(__half2(h));
  a = f.x * s;
  b = f.y * s;
}

// Bits of the smallest power of two s >= 2^-24 with amax / s <= 448 = 1.75 * 2^8.
__device__ __forceinline__ uint32_t scale_bits(uint32_t amax) {
  if (amax >= 0x7f800000u) return kNanBits;
  const int e = static_cast<int>(amax >> 23) - 8 + ((amax & 0x7fffffu) > 0x600000u ? 1 : 0);
  return max(e, 127 - 24) << 23;
}

// One team of kWarps warps per (sequence, block of tokens, head) the call touches.  A row of W
// codes is read by 2^lpr lanes, eight elements each; the team's rows follow one another over
// its lanes.  A thread keeps its first vectors in registers between the maximum and the
// encoding, and reads what is behind them a second time (from L1 or L2).  kSimple: one column a
// lane, at most kHold vectors and one page a block, which spares a third of the instructions
// (0.72 are issued a cycle: 8191 tokens of 8 x 256 bf16, B = 4, blocks of 64, 182 MB, take 35.5 us,
// 5.1 TB/s of 6.5 at the copy rate).
// kPages: pages are smaller than blocks of tokens, so each row is looked up (apart from the others since
// its code alone costs one token's write 0.4 us).
template <typename T, int kWarps, bool kSimple, bool kPages>
__global__ void __launch_bounds__(kThreads, 4)
kv_write_kernel(const KvGeom g, int n_new, uint32_t blocks_per_seq, const T* __restrict__ x, size_t x_stride, int lpr,
                const int32_t* __restrict__ start, const int32_t* __restrict__ count, int32_t* status) {
  using Raw = decltype(load8(static_cast<const T*>(nullptr)));
  constexpr int kHold = sizeof(T) == 2 ? 9 : 5;
  __shared__ uint32_t red[kThreads / 32];
  const int lane = threadIdx.x & 31, team_warp = (threadIdx.x >> 5) % kWarps;
  const uint32_t unit = blockIdx.x * (kThreads / 32 / kWarps) + (threadIdx.x >> 5) / kWarps;
  if (unit >= static_cast<uint32_t>(g.B) * blocks_per_seq * g.G) return;   // whole teams leave (a block-wide team has one unit)
  const uint32_t ub = g.G == 1 ? unit : unit / g.G;
  const int head = static_cast<int>(unit - ub * g.G);
  const int b = static_cast<int>(ub / blocks_per_seq), j = static_cast<int>(ub - b * blocks_per_seq);
  const int n = count != nullptr ? min(max(__ldg(count + b), 0), n_new) : n_new;
  const long long first = __ldg(start + b);
  const long long last = first + n;                              // one past the new tokens
  if (first < 0 || last > g.N) {
    if (j == 0 && head == 0 && lane == 0 && n > 0) raise_status(status, LSA_ERR_RANGE);
    if (first < 0) return;
  }
  const long long blk = (first >> g.block_log) + j;
  const long long t0 = blk << g.block_log;
  const int lo = static_cast<int>(max(t0, first) - first);       // new tokens of this block
  const int hi = static_cast<int>(min(min(t0 + (1ll << g.block_log), last), static_cast<long long>(g.N)) - first);
  if (hi <= lo) return;
  const int vpr = g.W / 8, rows = hi - lo;
  const int step_log = (kWarps == 8 ? 8 : 5) - lpr;              // rows of the team at a time
  const int row0 = (team_warp << (5 - lpr)) + (lane >> lpr), col0 = lane & ((1 << lpr) - 1);
  const T* xb = x + (static_cast<size_t>(b) * n_new + lo) * x_stride + static_cast<size_t>(head) * g.W;
  float* sp = g.scale + (static_cast<size_t>(b) * g.n_blocks + blk) * g.G + head;
  const bool grown_block = t0 < first;               // tokens before the new ones stay in the block
  const float before = grown_block ? *sp : 0.f;

  // The thread's vectors: rows row0, row0 + step, .. of column col0, then of column col0 + 32, ..
  const int nr = rows > row0 ? (rows - row0 + (1 << step_log) - 1) >> step_log : 0;
  const int nv = nr * (col0 < vpr ? (vpr - col0 + 31) >> 5 : 0);
  const size_t x_step = x_stride << step_log;
  const T* xp = xb + static_cast<size_t>(row0) * x_stride + col0 * 8;
  auto next_x = [&](int& left, const T*& p) {        // left: rows of this column from here on
    p += x_step;
    if (--left == 0) {
      left = nr;
      p += 256;
      p -= x_step * nr;
    }
  };
  Raw held[kHold];
  uint32_t m = 0;
  int left = nr;
  const T* p = xp;
#pragma unroll
  for (int k = 0; k < kHold; ++k)
    if (k < nv) {
      if constexpr (kSimple) {
        held[k] = load8(xp + k * x_step);
      } else {
        held[k] = load8(p);
        next_x(left, p);
      }
    }
  // Tokens that are not resident are skipped and have no part in the scale.
  const int t_new = static_cast<int>(first) + lo;    // the team's first token
  bool some = false;
  if constexpr (kPages) {
    bool away = false, here = false;
    for (int i = lane; i < rows; i += 32) (kv_row(g, b, t_new + i) < 0 ? away : here) = true;
    some = __any_sync(0xffffffffu, away);
    if (some) raise_status(status, LSA_ERR_RANGE);
    if (!__any_sync(0xffffffffu, here)) return;      // the whole team
  }
  auto counts = [&](int k) {                         // whether the row of the k-th vector does
    return !kPages || !some || kv_row(g, b, t_new + row0 + ((k % nr) << step_log)) >= 0;
  };
#pragma unroll
  for (int k = 0; k < kHold; ++k)
    if (k < nv && counts(k)) m = max(m, amax_bits(held[k]));
  for (int k = kHold; !kSimple && k < nv; ++k) {
    if (counts(k)) m = max(m, amax_bits(load8(p)));
    next_x(left, p);
  }
  m = __reduce_max_sync(0xffffffffu, m);
  if constexpr (kWarps > 1) {
    if (lane == 0) red[threadIdx.x / 32] = m;
    __syncthreads();                                 // and every thread has read the old scale
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) m = max(m, red[w]);
  } else {
    __syncwarp();
  }
  uint32_t sb = scale_bits(m);
  if (grown_block) {
    if (!(before <= 3.4e38f)) sb = kNanBits;
    else if (sb != kNanBits) sb = max(sb, __float_as_uint(max(before, 0.f)));
  }
  const float s = __uint_as_float(sb);
  const bool finite = sb != kNanBits;
  const float inv = finite ? 1.0f / s : 0.f;
  if (kPages && grown_block && !(before == s) && (finite || before == before)) {
    // The scale changes, which an earlier token that is not resident cannot follow: all stays as it is.
    bool away = false;
    for (long long t = t0 + lane; t < first; t += 32) away |= kv_row(g, b, static_cast<int>(t)) < 0;
    if (__any_sync(0xffffffffu, away)) {
      raise_status(status, LSA_ERR_RANGE);
      return;
    }
  }
  const long long place0 = kPages ? 0 : kv_row(g, b, t_new);
  if (place0 < 0) {
    raise_status(status, LSA_ERR_RANGE);
    return;
  }
  if (lane == 0 && team_warp == 0) *sp = s;

  const size_t row_bytes = static_cast<size_t>(g.G) * g.W;
  uint8_t* const base = g.rows + static_cast<size_t>(head) * g.W + col0 * 8;
  {
    uint8_t* dst = base + static_cast<size_t>(place0 + row0) * row_bytes;
    const size_t d_step = row_bytes << step_log;
    int r = row0, col = 0;
    auto put = [&](const Raw& raw) {
      bool there = true;
      if constexpr (kPages) {
        const long long place = kv_row(g, b, t_new + r);
        there = place >= 0;
        dst = base + static_cast<size_t>(there ? place : 0) * row_bytes + col;
      }
      if (there) {
        float f[8];
        to_floats(raw, f);
        *reinterpret_cast<uint2*>(dst) = finite ? encode8(f, inv) : make_uint2(0u, 0u);
      }
    };
    auto next_d = [&]() {
      dst += d_step;
      r += 1 << step_log;
      if (r >= rows) {
        r = row0;
        col += 256;
        dst += 256;
        dst -= d_step * nr;
      }
    };
    if constexpr (kSimple) {
#pragma unroll
      for (int k = 0; k < kHold; ++k)
        if (k < nv) {
          float f[8];
          to_floats(held[k], f);
          *reinterpret_cast<uint2*>(dst + k * d_step) = finite ? encode8(f, inv) : make_uint2(0u, 0u);
        }
    } else {
#pragma unroll
      for (int k = 0; k < kHold; ++k)
        if (k < nv) {
          put(held[k]);
          next_d();
        }
    }
    if (!kSimple && nv > kHold) {                                // from L1 or L2 again
      left = nr;
      p = xp;
      for (int k = 0; k < nv; ++k) {
        if (k >= kHold) {
          put(load8(p));
          next_d();
        }
        next_x(left, p);
      }
    }
  }
  if (grown_block && !(before == s)) {
    const float ratio = finite ? before * inv : 0.f;
    const int n_old = static_cast<int>(first - t0) * vpr;
    for (int v = team_warp * 32 + lane; v < n_old; v += kWarps * 32) {
      const int i = v / vpr;
      const long long row = kv_row(g, b, static_cast<int>(t0 + i));
      if (row < 0) continue;
      uint2* p = reinterpret_cast<uint2*>(g.rows + (static_cast<size_t>(row) * g.G + head) * g.W + (v - i * vpr) * 8);
      const uint2 code = *p;
      float f[8];
      decode2(code.x & 0xffffu, 1.f, f[0], f[1]);
      decode2(code.x >> 16, 1.f, f[2], f[3]);
      decode2(code.y & 0xffffu, 1.f, f[4], f[5]);
      decode2(code.y >> 16, 1.f, f[6], f[7]);
      *p = finite ? encode8(f, ratio) : make_uint2(0u, 0u);
    }
  }
}

__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// 32 bytes in one store.
__device__ __forceinline__ void store32(void* p, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}
__device__ __forceinline__ void store16(float* p, const float (&v)[16]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(v[8 * h + i]);
    store32(p + 8 * h, w);
  }
}
__device__ __forceinline__ void store16(__nv_bfloat16* p, const float (&v)[16]) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  store32(p, w);
}
// A warp reads 2^tpw_log listed tokens.  Its lanes look the tokens up first (list entry, page and,
// with one head, scale; the list's entry does not wait for the count), then take the tokens'
// rows together, kFlight vectors a lane in flight.  kWide: 16 codes a lane (32 bytes of bf16 out in
// one store) where the output's alignment allows it, else eight.  100 MB of listed 576-byte rows and
// their bf16 take 21.7 us (4.6 TB/s, 15.3 us at the copy rate; 23.5 with eight codes a lane), random rows
// as consecutive ones; more vectors in flight, or all 64 warps on an SM, change nothing.  What is left is the
// two dependent loads before a warp's rows, and that two thirds of the bytes are stores.
template <typename T, bool kWide>
__global__ void __launch_bounds__(kThreads)
kv_read_kernel(const KvGeom g, const int32_t* __restrict__ idx, int cap, const int32_t* __restrict__ count,
               T* __restrict__ out, int32_t* status, uint32_t warps_per_seq, int tpw_log) {
  constexpr int V = kWide ? 16 : 8;
  using Code = std::conditional_t<kWide, uint4, uint2>;
  const uint32_t vpr = g.W / V, vpt = g.G * vpr;   // vectors of a row and of a token
  const uint32_t warp = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  const uint32_t b = warp / warps_per_seq;
  if (b >= static_cast<uint32_t>(g.B)) return;
  const int j0 = static_cast<int>((warp - b * warps_per_seq) << tpw_log);
  int tok = -1, row = -1;
  if (lane < (1u << tpw_log) && j0 + static_cast<int>(lane) < cap)
    tok = idx != nullptr ? __ldg(idx + static_cast<size_t>(b) * cap + j0 + lane) : j0 + static_cast<int>(lane);
  const int n = count != nullptr ? min(max(__ldg(count + b), 0), cap) : cap;
  const int mine = min(1 << tpw_log, n - j0);      // tokens of this warp; what lies behind the count is left alone
  if (mine <= 0) return;
  float scale = 0.f;
  if (static_cast<int>(lane) < mine) {
    if (tok >= 0) {
      if (tok < g.N) {
        scale = __ldg(g.scale + kv_scale_at(g, b, tok, 0));
        row = static_cast<int>(kv_row(g, b, tok));
      }
      if (row < 0) raise_status(status, LSA_ERR_RANGE);
    }
  }
  T* const to = out + (static_cast<size_t>(b) * cap + j0) * vpt * V + lane * V;
  const uint32_t total = mine * vpt;
  uint32_t tk = 0, c = lane;                       // token of this lane's vector, and the vector in it
  while (c >= vpt) { c -= vpt; ++tk; }
  for (uint32_t v0 = 0; v0 < total; v0 += 32 * kFlight) {
    Code code[kFlight];
    float s[kFlight];
    bool there[kFlight];
#pragma unroll
    for (int k = 0; k < kFlight; ++k) {
      const int from = min(tk, 31u);
      const int r = __shfl_sync(0xffffffffu, row, from);
      s[k] = __shfl_sync(0xffffffffu, scale, from);
      const int t = __shfl_sync(0xffffffffu, tok, from);
      there[k] = v0 + k * 32 + lane < total && r >= 0;
      if (there[k]) {
        if (g.G > 1) s[k] = __ldg(g.scale + kv_scale_at(g, b, t, c / vpr));
        code[k] = __ldg(reinterpret_cast<const Code*>(g.rows + (static_cast<size_t>(r) * vpt + c) * V));
      }
      c += 32;
      while (c >= vpt) { c -= vpt; ++tk; }
    }
#pragma unroll
    for (int k = 0; k < kFlight; ++k) {
      if (!there[k]) continue;
      const uint32_t* w = reinterpret_cast<const uint32_t*>(&code[k]);
      float f[V];
#pragma unroll
      for (int i = 0; i < V / 2; ++i) decode2((w[i / 2] >> (i % 2 * 16)) & 0xffffu, s[k], f[2 * i], f[2 * i + 1]);
      if constexpr (kWide) store16(to + static_cast<size_t>(v0 + k * 32) * V, f);
      else store8(to + static_cast<size_t>(v0 + k * 32) * V, f);
    }
  }
}

template <typename T>
void write_typed(const KvGeom& g, int n_new, int per_seq, const void* x, size_t x_stride, const int32_t* start,
                 const int32_t* count, int32_t* status, cudaStream_t s) {
  const long long units = static_cast<long long>(g.B) * per_seq * g.G;
  const int vpr = g.W / 8, rows = std::min(1 << g.block_log, n_new);
  int lpr = 0;
  while (lpr < 5 && (1 << lpr) < vpr) ++lpr;
  // A warp takes a unit whose vectors its lanes can hold, a block of eight warps a larger one.
  const int per_lane = ((rows << lpr) + 31) / 32 * ((vpr + 31) / 32);
  const int hold = sizeof(T) == 2 ? 9 : 5, team_lane = ((rows << lpr) + 255) / 256;   // vectors a lane of eight warps, one column
  const bool simple = vpr <= 32;
  const unsigned small = static_cast<unsigned>((units + 7) / 8), large = static_cast<unsigned>(units);
  const T* xt = static_cast<const T*>(x);
  const bool pages = g.page_log < g.block_log;
  auto launch = [&](auto kern, unsigned grid) {
    kern<<<grid, kThreads, 0, s>>>(g, n_new, per_seq, xt, x_stride, lpr, start, count, status);
  };
  if (per_lane <= hold) {
    launch(pages ? kv_write_kernel<T, 1, false, true> : simple ? kv_write_kernel<T, 1, true, false> : kv_write_kernel<T, 1, false, false>, small);
  } else {
    launch(pages ? kv_write_kernel<T, 8, false, true>
                 : team_lane <= hold && simple ? kv_write_kernel<T, 8, true, false> : kv_write_kernel<T, 8, false, false>, large);
  }
}

}  // namespace

int launch_kv_write(const KvGeom& g, int T, int xdt, const void* x, size_t x_stride, const int32_t* start,
                    const int32_t* count, int32_t* status, cudaStream_t s) {
  const int block = 1 << g.block_log;
  const int per_seq = static_cast<int>((static_cast<long long>(T) + 2 * block - 2) / block);
  if (xdt == LSA_F32) write_typed<float>(g, T, per_seq, x, x_stride, start, count, status, s);
  else write_typed<__nv_bfloat16>(g, T, per_seq, x, x_stride, start, count, status, s);
  return check_launch("kv_write");
}

int launch_kv_read(const KvGeom& g, const int32_t* idx, int cap, const int32_t* count, int odt, void* out,
                   int32_t* status, cudaStream_t s) {
  // As many tokens a warp (up to 4) as leave 64 warps for each SM (those rows: the same with 4 tokens a
  // warp and with 8, 2.8 us more with 2).
  int tpw = 0;
  while (tpw < 2 && (static_cast<long long>(g.B) * cap >> (tpw + 1)) >= 64 * 148) ++tpw;
  const long long per_seq = (cap + (1ll << tpw) - 1) >> tpw, warps = per_seq * g.B;
  if (warps > 0x7fffffffll || static_cast<long long>(g.G) * (g.W / 8) > (1 << 24))
    return fail(LSA_ERR_UNSUPPORTED, "kv_read: B * cap = %lld, G * W = %lld (at most 2^31, 2^27)", static_cast<long long>(g.B) * cap, static_cast<long long>(g.G) * g.W);
  const unsigned grid = static_cast<unsigned>((warps + kThreads / 32 - 1) / (kThreads / 32)), ps = static_cast<unsigned>(per_seq);
  const bool wide = aligned(out, 32);              // rows are multiples of 16 codes
  if (odt == LSA_F32) {
    if (wide) kv_read_kernel<float, true><<<grid, kThreads, 0, s>>>(g, idx, cap, count, static_cast<float*>(out), status, ps, tpw);
    else kv_read_kernel<float, false><<<grid, kThreads, 0, s>>>(g, idx, cap, count, static_cast<float*>(out), status, ps, tpw);
  } else {
    if (wide) kv_read_kernel<__nv_bfloat16, true><<<grid, kThreads, 0, s>>>(g, idx, cap, count, static_cast<__nv_bfloat16*>(out), status, ps, tpw);
    else kv_read_kernel<__nv_bfloat16, false><<<grid, kThreads, 0, s>>>(g, idx, cap, count, static_cast<__nv_bfloat16*>(out), status, ps, tpw);
  }
  return check_launch("kv_read");
}

}  // namespace lsa
