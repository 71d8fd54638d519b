// Rotary positions of part of a head.
//
// Pair i of a head turns by the angle pos * freq[i]: (u, v) -> m (u cos a - v sin a,
// u sin a + v cos a), m a magnitude factor.  The map is a rotation times m, so its gradient is
// the same rotation by -a times m: the inverse call on the output's gradient.
//
// Positions reach 2^20 and more, where an fp32 product pos * freq is off by hundredths of a
// radian, so the angle is formed in fp64, in turns, and only its fraction of a turn is
// rounded to fp32 (error 2^-25 of a turn).  Sine and cosine are computed once per token and
// pair and shared by the token's heads.
#include <algorithm>

#include "kv_common.cuh"

namespace lsa {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float get(const float* p) { return *p; }
__device__ __forceinline__ float get(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void set(float* p, float v) { *p = v; }
__device__ __forceinline__ void set(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

template <typename T>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeArgs a) {
  extern __shared__ float2 cs[];                    // [rot / 2] of the block's token
  const int np = a.rot / 2;
  for (long long r = blockIdx.x; r < a.R; r += gridDim.x) {
    const double pos = static_cast<double>(__ldg(a.pos + r)) * (a.inverse ? -1.0 : 1.0);
    __syncthreads();
    for (int i = threadIdx.x; i < np; i += kThreads) {
      const double turns = pos * __ldg(a.freq + i) * 0.15915494309189533576888;   // 1 / (2 pi)
      float si, co;
      sincospif(2.0f * static_cast<float>(turns - rint(turns)), &si, &co);
      cs[i] = make_float2(co * a.mscale, si * a.mscale);
    }
    __syncthreads();
    const T* x = static_cast<const T*>(a.x) + r * a.x_token;
    T* o = static_cast<T*>(a.out) + r * a.o_token;
    for (int e = threadIdx.x; e < a.H * np; e += kThreads) {
      const int h = e / np, i = e - h * np;
      const int iu = a.half ? i : 2 * i, iv = a.half ? i + np : 2 * i + 1;
      const float u = get(x + h * a.x_head + iu), v = get(x + h * a.x_head + iv);
      const float2 c = cs[i];
      set(o + h * a.o_head + iu, u * c.x - v * c.y);
      set(o + h * a.o_head + iv, u * c.y + v * c.x);
    }
  }
}

}  // namespace

int launch_rope(const RopeArgs& a, cudaStream_t s) {
  const unsigned grid = static_cast<unsigned>(std::min(a.R, 1 << 20));
  const size_t smem = static_cast<size_t>(a.rot / 2) * sizeof(float2);
  if (a.dt == LSA_F32) rope_kernel<float><<<grid, kThreads, smem, s>>>(a);
  else rope_kernel<__nv_bfloat16><<<grid, kThreads, smem, s>>>(a);
  return check_launch("rope");
}

}  // namespace lsa
