// Rotary positions of part of a head.
//
// Pair i of a head turns by the angle pos * freq[i]: (u, v) -> m (u cos a - v sin a,
// u sin a + v cos a), m a magnitude factor.  The map is a rotation times m, so its gradient is
// the same rotation by -a times m: the inverse call on the output's gradient.
//
// Positions reach 2^20 and more, where an fp32 product pos * freq is off by hundredths of a
// radian, so the angle is formed in fp64, in turns, and only its fraction of a turn is
// rounded to fp32 (error 2^-25 of a turn).
//
// Each element is read and written once, so memory bounds the kernel.  A block takes several
// tokens at a time: first its threads compute the tokens' sines and cosines into shared memory
// (shared by all heads), then each thread moves 16-byte vectors, two in flight for each pair
// of halves.  Rows whose base, strides or width do not allow 16 bytes go pair by pair.  16384
// tokens of 32 heads of 128 bf16 (268 MB) take 46.4 us, 5.8 TB/s; 32-byte vectors make it 47.6.
#include <algorithm>

#include "kv_common.cuh"

namespace lsa {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float get(const float* p) { return *p; }
__device__ __forceinline__ float get(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void set(float* p, float v) { *p = v; }
__device__ __forceinline__ void set(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// 16 bytes as floats and back.
__device__ __forceinline__ void unpack(uint4 r, float (&v)[4]) {
  v[0] = __uint_as_float(r.x); v[1] = __uint_as_float(r.y); v[2] = __uint_as_float(r.z); v[3] = __uint_as_float(r.w);
}
__device__ __forceinline__ void unpack(uint4 r, float (&v)[8]) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 packed(const float (&v)[4]) {
  return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
}
__device__ __forceinline__ uint4 packed(const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// kVec: 16-byte vectors of V elements; items of a head: np / V pairs of vectors (half layout) or
// rot / V vectors (interleaved).  Without kVec an item is one pair.
template <typename T, bool kVec, bool kHalf>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeArgs a, int tokens) {
  extern __shared__ float2 cs[];                    // [tokens][rot / 2]: m cos, m sin
  constexpr int V = 16 / sizeof(T);
  const int np = a.rot / 2;
  const uint32_t per_head = kVec ? (kHalf ? np / V : a.rot / V) : np;
  for (long long r0 = static_cast<long long>(blockIdx.x) * tokens; r0 < a.R; r0 += static_cast<long long>(gridDim.x) * tokens) {
    const int nt = static_cast<int>(min(static_cast<long long>(tokens), a.R - r0));
    __syncthreads();
    for (uint32_t e = threadIdx.x; e < static_cast<uint32_t>(nt * np); e += kThreads) {
      const uint32_t t = e / np, i = e - t * np;
      const double pos = static_cast<double>(__ldg(a.pos + r0 + t)) * (a.inverse ? -1.0 : 1.0);
      const double turns = pos * __ldg(a.freq + i) * 0.15915494309189533576888;   // 1 / (2 pi)
      float si, co;
      sincospif(2.0f * static_cast<float>(turns - rint(turns)), &si, &co);
      cs[e] = make_float2(co * a.mscale, si * a.mscale);
    }
    __syncthreads();
    const uint32_t per_token = a.H * per_head, items = nt * per_token;
#pragma unroll 2
    for (uint32_t e = threadIdx.x; e < items; e += kThreads) {
      const uint32_t t = nt == 1 ? 0 : e / per_token, f = e - t * per_token;
      const uint32_t h = f / per_head, i = f - h * per_head;
      const T* x = static_cast<const T*>(a.x) + (r0 + t) * a.x_token + h * a.x_head;
      T* o = static_cast<T*>(a.out) + (r0 + t) * a.o_token + h * a.o_head;
      const float2* c = cs + t * np;
      if constexpr (!kVec) {
        const int iu = kHalf ? i : 2 * i, iv = kHalf ? i + np : 2 * i + 1;
        const float u = get(x + iu), v = get(x + iv);
        set(o + iu, u * c[i].x - v * c[i].y);
        set(o + iv, u * c[i].y + v * c[i].x);
      } else if constexpr (kHalf) {
        const uint4 ru = *reinterpret_cast<const uint4*>(x + i * V), rv = *reinterpret_cast<const uint4*>(x + np + i * V);
        float u[V], v[V], p[V], q[V];
        unpack(ru, u);
        unpack(rv, v);
#pragma unroll
        for (int k = 0; k < V; ++k) {
          const float2 w = c[i * V + k];
          p[k] = u[k] * w.x - v[k] * w.y;
          q[k] = u[k] * w.y + v[k] * w.x;
        }
        *reinterpret_cast<uint4*>(o + i * V) = packed(p);
        *reinterpret_cast<uint4*>(o + np + i * V) = packed(q);
      } else {
        float u[V], p[V];
        unpack(*reinterpret_cast<const uint4*>(x + i * V), u);
#pragma unroll
        for (int k = 0; k < V / 2; ++k) {
          const float2 w = c[i * (V / 2) + k];
          p[2 * k] = u[2 * k] * w.x - u[2 * k + 1] * w.y;
          p[2 * k + 1] = u[2 * k] * w.y + u[2 * k + 1] * w.x;
        }
        *reinterpret_cast<uint4*>(o + i * V) = packed(p);
      }
    }
  }
}

template <typename T>
void rope_typed(const RopeArgs& a, cudaStream_t s) {
  constexpr int V = 16 / sizeof(T);
  const bool vec = aligned(a.x, 16) && aligned(a.out, 16) && a.x_token % V == 0 && a.x_head % V == 0 &&
                   a.o_token % V == 0 && a.o_head % V == 0 && a.rot % (a.half ? 2 * V : V) == 0;
  // Tokens of a block: enough vectors for each thread to move four (fewer tokens when there
  // are too few for every SM), at most 48 KB of sines.
  const long long per_token = std::max<long long>(1, static_cast<long long>(a.H) * a.rot / (vec ? (a.half ? 2 * V : V) : 2));
  long long tokens = std::max<long long>(1, 4 * kThreads / per_token);
  tokens = std::min<long long>({tokens, std::max(1, a.R / (4 * 148)), 6144 / std::max(1, a.rot / 2)});
  tokens = std::max<long long>(1, tokens);
  const unsigned grid = static_cast<unsigned>(std::min<long long>((a.R + tokens - 1) / tokens, 1 << 30));
  const size_t smem = static_cast<size_t>(tokens) * (a.rot / 2) * sizeof(float2);
  const int t = static_cast<int>(tokens);
  if (vec && a.half) rope_kernel<T, true, true><<<grid, kThreads, smem, s>>>(a, t);
  else if (vec) rope_kernel<T, true, false><<<grid, kThreads, smem, s>>>(a, t);
  else if (a.half) rope_kernel<T, false, true><<<grid, kThreads, smem, s>>>(a, t);
  else rope_kernel<T, false, false><<<grid, kThreads, smem, s>>>(a, t);
}

}  // namespace

int launch_rope(const RopeArgs& a, cudaStream_t s) {
  if (a.dt == LSA_F32) rope_typed<float>(a, s);
  else rope_typed<__nv_bfloat16>(a, s);
  return check_launch("rope");
}

}  // namespace lsa
