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

#include "kv_common.cuh"

namespace lsa {
namespace {

constexpr int kThreads = 256;
constexpr int kHold = 8;        // 8-element vectors a thread keeps in registers between the passes
constexpr uint32_t kNanBits = 0x7fc00000u;

// Eight consecutive elements as fp32 bits.
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
  const uint4 a = __ldg(reinterpret_cast<const uint4*>(p));
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
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

// Largest magnitude as its bits: non-finite values have the largest of all.
__device__ __forceinline__ uint32_t amax_bits(const float (&v)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
  return m;
}

// Bits of the smallest power of two s >= 2^-24 with amax / s <= 448 = 1.75 * 2^8.
__device__ __forceinline__ uint32_t scale_bits(uint32_t amax) {
  if (amax >= 0x7f800000u) return kNanBits;
  const int e = static_cast<int>(amax >> 23) - 8 + ((amax & 0x7fffffu) > 0x600000u ? 1 : 0);
  return max(e, 127 - 24) << 23;
}

// One team of kTeam threads per (sequence, block of tokens, head) the call touches.
template <typename T, int kTeam>
__global__ void __launch_bounds__(kThreads)
kv_write_kernel(const KvGeom g, int n_new, int blocks_per_seq, const T* __restrict__ x, size_t x_stride,
                const int32_t* __restrict__ start, const int32_t* __restrict__ count, int32_t* status) {
  __shared__ uint32_t red[kThreads / 32];
  const int lane = threadIdx.x % kTeam;
  const long long unit = static_cast<long long>(blockIdx.x) * (kThreads / kTeam) + threadIdx.x / kTeam;
  const long long units = static_cast<long long>(g.B) * blocks_per_seq * g.G;
  if (unit >= units) return;           // whole teams leave (a block-wide team has one unit)
  const int head = static_cast<int>(unit % g.G);
  const long long ub = unit / g.G;
  const int b = static_cast<int>(ub / blocks_per_seq), j = static_cast<int>(ub % blocks_per_seq);
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
  const int vpr = g.W / 8;
  const int nv = (hi - lo) * vpr;
  const T* xb = x + (static_cast<size_t>(b) * n_new + lo) * x_stride + static_cast<size_t>(head) * g.W;
  auto src = [&](int v) { const int i = v / vpr; return xb + static_cast<size_t>(i) * x_stride + (v - i * vpr) * 8; };

  float held[kHold][8];
  uint32_t m = 0;
#pragma unroll
  for (int k = 0; k < kHold; ++k) {
    const int v = lane + k * kTeam;
    if (v < nv) {
      load8(src(v), held[k]);
      m = max(m, amax_bits(held[k]));
    }
  }
  for (int v = lane + kHold * kTeam; v < nv; v += kTeam) {
    float f[8];
    load8(src(v), f);
    m = max(m, amax_bits(f));
  }
  m = __reduce_max_sync(0xffffffffu, m);
  if constexpr (kTeam > 32) {
    if ((threadIdx.x & 31) == 0) red[threadIdx.x / 32] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) m = max(m, red[w]);
  }
  uint32_t sb = scale_bits(m);
  float* sp = g.scale + (static_cast<size_t>(b) * g.n_blocks + blk) * g.G + head;
  const bool grown_block = t0 < first;               // tokens before the new ones stay in the block
  float before = 0.f;
  if (grown_block) {
    before = *sp;
    if (!(before <= 3.4e38f)) sb = kNanBits;
    else if (sb != kNanBits) sb = max(sb, __float_as_uint(max(before, 0.f)));
    if constexpr (kTeam > 32) __syncthreads(); else __syncwarp();   // every thread has read the old scale
  }
  const float s = __uint_as_float(sb);
  const bool finite = sb != kNanBits;
  const float inv = finite ? 1.0f / s : 0.f;
  if (lane == 0) *sp = s;

  auto put = [&](int v, const float (&f)[8]) {
    const int i = v / vpr;
    const long long row = kv_row(g, b, static_cast<int>(first + lo + i));
    if (row < 0) {
      raise_status(status, LSA_ERR_RANGE);
      return;
    }
    const uint2 code = finite ? encode8(f, inv) : make_uint2(0u, 0u);
    *reinterpret_cast<uint2*>(g.rows + (static_cast<size_t>(row) * g.G + head) * g.W + (v - i * vpr) * 8) = code;
  };
#pragma unroll
  for (int k = 0; k < kHold; ++k) {
    const int v = lane + k * kTeam;
    if (v < nv) put(v, held[k]);
  }
  for (int v = lane + kHold * kTeam; v < nv; v += kTeam) {
    float f[8];
    load8(src(v), f);
    put(v, f);
  }
  if (grown_block && !(before == s)) {
    const float ratio = finite ? before * inv : 0.f;
    const int n_old = static_cast<int>(first - t0) * vpr;
    for (int v = lane; v < n_old; v += kTeam) {
      const int i = v / vpr;
      const long long row = kv_row(g, b, static_cast<int>(t0 + i));
      if (row < 0) continue;
      uint2* p = reinterpret_cast<uint2*>(g.rows + (static_cast<size_t>(row) * g.G + head) * g.W + (v - i * vpr) * 8);
      const uint2 c = *p;
      float f[8];
      decode2(c.x & 0xffffu, 1.f, f[0], f[1]);
      decode2(c.x >> 16, 1.f, f[2], f[3]);
      decode2(c.y & 0xffffu, 1.f, f[4], f[5]);
      decode2(c.y >> 16, 1.f, f[6], f[7]);
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

// Thread per eight codes of one listed token's rows.
template <typename T>
__global__ void __launch_bounds__(kThreads)
kv_read_kernel(const KvGeom g, const int32_t* __restrict__ idx, int cap, const int32_t* __restrict__ count,
               T* __restrict__ out, int32_t* status) {
  const int vpt = g.G * (g.W / 8);                 // vectors of one token
  const long long per_seq = static_cast<long long>(cap) * vpt, all = per_seq * g.B;
  for (long long i = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x; i < all;
       i += static_cast<long long>(gridDim.x) * kThreads) {
    const int b = static_cast<int>(i / per_seq);
    const long long r = i - b * per_seq;
    const int j = static_cast<int>(r / vpt), v = static_cast<int>(r - static_cast<long long>(j) * vpt);
    if (count != nullptr && j >= __ldg(count + b)) continue;
    const int t = idx != nullptr ? __ldg(idx + static_cast<size_t>(b) * cap + j) : j;
    if (t < 0) continue;
    const long long row = t < g.N ? kv_row(g, b, t) : -1;
    if (row < 0) {
      raise_status(status, LSA_ERR_RANGE);
      continue;
    }
    const int head = v / (g.W / 8);
    const float s = __ldg(g.scale + kv_scale_at(g, b, t, head));
    const uint2 c = *reinterpret_cast<const uint2*>(g.rows + static_cast<size_t>(row) * g.G * g.W + v * 8);
    float f[8];
    decode2(c.x & 0xffffu, s, f[0], f[1]);
    decode2(c.x >> 16, s, f[2], f[3]);
    decode2(c.y & 0xffffu, s, f[4], f[5]);
    decode2(c.y >> 16, s, f[6], f[7]);
    store8(out + static_cast<size_t>(i) * 8, f);
  }
}

template <typename T>
void write_typed(const KvGeom& g, int n_new, int per_seq, const void* x, size_t x_stride, const int32_t* start,
                 const int32_t* count, int32_t* status, cudaStream_t s) {
  const long long units = static_cast<long long>(g.B) * per_seq * g.G;
  const long long vectors = (static_cast<long long>(std::min(1 << g.block_log, n_new))) * (g.W / 8);
  // A warp keeps up to 256 vectors of its unit in registers; larger units get a whole block.
  if (vectors <= 32 * kHold) {
    kv_write_kernel<T, 32><<<static_cast<unsigned>((units + 7) / 8), kThreads, 0, s>>>(
        g, n_new, per_seq, static_cast<const T*>(x), x_stride, start, count, status);
  } else {
    kv_write_kernel<T, kThreads><<<static_cast<unsigned>(units), kThreads, 0, s>>>(
        g, n_new, per_seq, static_cast<const T*>(x), x_stride, start, count, status);
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
  const long long all = static_cast<long long>(g.B) * cap * g.G * (g.W / 8);
  const unsigned grid = static_cast<unsigned>(std::min<long long>((all + kThreads - 1) / kThreads, 1 << 30));
  if (odt == LSA_F32) kv_read_kernel<float><<<grid, kThreads, 0, s>>>(g, idx, cap, count, static_cast<float*>(out), status);
  else kv_read_kernel<__nv_bfloat16><<<grid, kThreads, 0, s>>>(g, idx, cap, count, static_cast<__nv_bfloat16*>(out), status);
  return check_launch("kv_read");
}

}  // namespace lsa
