// Attention over the 8-bit KV cache on the CUDA cores, and the join of a sequence's parts.
//
// For a query column c (a query token and head of one KV head's group) over the visible
// tokens t:  x_t = sm * scale_t * (q_c . k_t),  o_c = sum_t 2^(x_t log2 e - m) scale_t v_t / l_c,
// l_c = sum_t 2^(x_t log2 e - m), with k and v the stored codes.  One pass: the running
// maximum m, the sum l and the weighted values are rescaled when a tile raises m.
//
// What bounds it: for short calls the latency of a tile's steps (8 columns over 64 listed tokens of
// 576 codes, one sequence: 8.5 us; 21.8 with a warp a column and nothing read ahead); for long ones
// shared memory, which a column's products read at four bytes a multiply-add (16384 tokens x 16 columns,
// B = 4: 164 us).
//
// This path serves fp32 queries (which the tensor cores would round) and row shapes the
// tensor-core path declines; products, sums and statistics are fp32.  Tokens are split into
// parts when there are few (sequence, KV head) units; the parts' unnormalised sums are joined
// by the second kernel.
#include <algorithm>

#include "kv_common.cuh"

namespace lsa {
namespace {

constexpr int kTile = 32;          // tokens of a tile: one per lane for the scores
constexpr int kWarps = 8;          // one, two, four or all of them for a column
constexpr int kWords = 5;          // words of a row a lane reads ahead (640 codes; 8 of them cost a tenth more)
constexpr int kMaxVpl = 16;        // value columns per lane of one warp (dv <= 512)

__device__ __forceinline__ void store_out(void* out, int qdt, size_t i, float v) {
  if (qdt == LSA_F32) static_cast<float*>(out)[i] = v;
  else static_cast<__nv_bfloat16*>(out)[i] = __float2bfloat16_rn(v);
}

// Four codes as floats.
__device__ __forceinline__ void decode4(uint32_t c, float* to) {
  const float2 lo = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(c & 0xffffu), __NV_E4M3)));
  const float2 hi = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(c >> 16), __NV_E4M3)));
  *reinterpret_cast<float4*>(to) = make_float4(lo.x, lo.y, hi.x, hi.y);
}

// kVec: value columns start and end on multiples of four, so that a lane holds neighbouring
// ones (16-byte shared loads, 8-byte ones in a team of eight); else every 32nd.
//
// kTeam warps work on a column: each sums its share of the score's products, the shares
// are added in one order through shared memory, and each holds its share of the value columns.
//
// Reading a token takes a chain of loads (list entry, page and scale, row); tiles pass through it
// in four steps, so that a step's loads are in flight while the tile before is multiplied: the
// entry is read three tiles ahead, page and scale two, the row's codes one, into registers.
template <bool kVec, int kTeam>
__global__ void __launch_bounds__(kWarps * 32, 2)
kv_attend_simt_kernel(const KvAttendArgs a, int col_blocks, int rows_used) {
  constexpr int kCols = kWarps / kTeam;            // columns of a block
  constexpr int kAcc = kMaxVpl / kTeam;            // value columns of a lane
  constexpr int kRun = !kVec ? 1 : kAcc < 4 ? kAcc : 4;   // neighbouring ones
  extern __shared__ __align__(16) float smem[];
  const KvGeom& g = a.g;
  const int pitch = (rows_used + 31) / 32 * 32 + 4;   // a lane per token reads 16 bytes without conflicts
  const int dpad = (a.d + 3) & ~3;
  float* kv = smem;                                // [kTile][pitch] values without their scale
  float* qs = kv + kTile * pitch;                  // [kCols][dpad]
  float* ps = qs + kCols * dpad;                   // [kWarps][kTile] weights times scales
  float* red = ps + kWarps * kTile;                // [kWarps][kTile] shares of the scores
  const int hg = a.H / g.G, ncol = a.Tq * hg;
  uint32_t u = blockIdx.x;
  const int part = static_cast<int>(u % a.splits); u /= a.splits;
  const int cb = static_cast<int>(u % col_blocks); u /= col_blocks;
  const int head = static_cast<int>(u % g.G), b = static_cast<int>(u / g.G);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int mine = warp / kTeam, share = warp % kTeam;
  const KvSpan sp = kv_span(a, b);
  const int tiles = (sp.total + kTile - 1) / kTile;
  const int tile0 = static_cast<int>(static_cast<long long>(tiles) * part / a.splits);
  const int tile1 = static_cast<int>(static_cast<long long>(tiles) * (part + 1) / a.splits);
  const int col = cb * kCols + mine, cc = min(col, ncol - 1), qi = cc / hg;
  const int wpr = rows_used / 4;                   // 4-code words of a row
  constexpr int kRows = kTile / kWarps;

  // The steps of a tile.  Every warp takes them for all 32 tokens, a token a lane.
  auto entry_of = [&](int tile) -> int {           // the token, unchecked; -1: an empty place
    const int v = tile * kTile + lane;
    if (tile >= tile1 || v >= sp.total) return -1;
    bool main = true;
    return v < sp.n_main ? kv_token(a, sp, b, v, main) : a.idx[static_cast<size_t>(b) * a.cap + (v - sp.n_main)];
  };
  auto place_of = [&](int& t, int& page, float& s) {
    if (t >= sp.len) {                             // only a list entry can be
      raise_status(a.status, LSA_ERR_RANGE);
      t = -1;
    }
    t = max(t, -1);
    page = t >= 0 ? kv_page(g, b, t) : -1;
    s = t >= 0 ? g.scale[kv_scale_at(g, b, t, head)] : 0.f;
  };
  uint32_t code[kRows][kWords];
  int row = -1;                                    // of the lane's token
  auto from = [&](int k) {                         // the warp's k-th row, or null
    const int r = __shfl_sync(0xffffffffu, row, warp + k * kWarps);
    return r < 0 ? nullptr : reinterpret_cast<const uint32_t*>(g.rows + (static_cast<size_t>(r) * g.G + head) * g.W);
  };
  auto codes_of = [&](int& t, int page) {          // a warp every kWarps-th row
    row = t >= 0 ? static_cast<int>(kv_row_of(g, b, t, page)) : -1;
    if (t >= 0 && row < 0) {
      raise_status(a.status, LSA_ERR_RANGE);
      t = -1;
    }
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      const uint32_t* src = from(k);
#pragma unroll
      for (int j = 0; j < kWords; ++j) {
        const int i = lane + 32 * j;
        code[k][j] = src != nullptr && i < wpr ? src[i] : 0u;
      }
    }
  };
  int t1 = entry_of(tile0), t2 = entry_of(tile0 + 1), t3 = entry_of(tile0 + 2), page1, page2;
  float s1, s2;
  place_of(t1, page1, s1);
  {
    const size_t at = ((static_cast<size_t>(b) * a.Tq + qi) * a.H + head * hg + (cc - qi * hg)) * a.d;
    for (int e = share * 32 + lane; e < dpad; e += 32 * kTeam) {
      float v = 0.f;
      if (e < a.d) v = a.qdt == LSA_F32 ? static_cast<const float*>(a.q)[at + e] : __bfloat162float(static_cast<const __nv_bfloat16*>(a.q)[at + e]);
      qs[mine * dpad + e] = v;
    }
  }
  codes_of(t1, page1);
  place_of(t2, page2, s2);
  float acc[kAcc], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int k = 0; k < kAcc; ++k) acc[k] = 0.f;
  // value column of accumulator k
  auto vcol = [&](int k) { return ((k / kRun) * kTeam + share) * 32 * kRun + lane * kRun + k % kRun; };
  const int pos = sp.len - a.Tq + qi;
  const float xs = a.sm * 1.44269504088896f;       // log2 e
  const int dq = dpad / 4, d0 = dq * share / kTeam, d1 = dq * (share + 1) / kTeam;
  for (int tile = tile0; tile < tile1; ++tile) {
    __syncthreads();                               // the tile before is used up
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      float* to = kv + (warp + k * kWarps) * pitch;
#pragma unroll
      for (int j = 0; j < kWords; ++j)
        if (lane + 32 * j < wpr) decode4(code[k][j], to + 4 * (lane + 32 * j));
      if (wpr > 32 * kWords) {                     // the rest of a wide row is not read ahead
        const uint32_t* src = from(k);
        for (int i = lane + 32 * kWords; i < wpr; i += 32) decode4(src != nullptr ? src[i] : 0u, to + 4 * i);
      }
    }
    const int tok = t1;
    const float s = s1;
    const bool listed = tile * kTile + lane >= sp.n_main;
    t1 = t2;
    s1 = s2;
    codes_of(t1, page2);
    t2 = t3;
    place_of(t2, page2, s2);
    t3 = entry_of(tile + 3);
    __syncthreads();
    float4 x4 = make_float4(0.f, 0.f, 0.f, 0.f);
    const float4* kr = reinterpret_cast<const float4*>(kv + lane * pitch);
    const float4* qr = reinterpret_cast<const float4*>(qs + mine * dpad);
#pragma unroll 4
    for (int k = d0; k < d1; ++k) {
      const float4 kk = kr[k], q = qr[k];
      x4.x = fmaf(q.x, kk.x, x4.x);
      x4.y = fmaf(q.y, kk.y, x4.y);
      x4.z = fmaf(q.z, kk.z, x4.z);
      x4.w = fmaf(q.w, kk.w, x4.w);
    }
    float dot = (x4.x + x4.y) + (x4.z + x4.w);
    if constexpr (kTeam > 1) {
      red[warp * kTile + lane] = dot;
      __syncthreads();
      dot = 0.f;
#pragma unroll
      for (int k = 0; k < kTeam; ++k) dot += red[(mine * kTeam + k) * kTile + lane];
    }
    bool see = tok >= 0;
    if (see) see = listed != kv_sees(a, tok, pos);  // a list entry that the window has is seen there
    const float x = see ? dot * (xs * s) : -INFINITY;
    float tm = x;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) tm = fmaxf(tm, __shfl_xor_sync(0xffffffffu, tm, o));
    const float mn = fmaxf(m, tm);
    const float ref = mn == -INFINITY ? 0.f : mn;
    const float f = exp2f(m - ref);                // 0 while nothing has been seen
    float p = see ? exp2f(x - ref) : 0.f;
    if (see && !(s <= 3.4e38f)) p = __int_as_float(0x7fc00000);   // a block marked non-finite makes the result NaN
    m = mn;
    float sum = p;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    l = l * f + sum;
    ps[warp * kTile + lane] = see ? p * s : 0.f;
    __syncwarp();
#pragma unroll
    for (int k = 0; k < kAcc; ++k) acc[k] *= f;
#pragma unroll 4
    for (int t = 0; t < kTile; ++t) {
      const float w = ps[warp * kTile + t];
      const float* vr = kv + t * pitch + a.voff;
#pragma unroll
      for (int k = 0; k < kAcc; k += kRun)
        if (vcol(k) < a.dv) {
          float v[kRun];
          if constexpr (kRun == 4) *reinterpret_cast<float4*>(v) = *reinterpret_cast<const float4*>(vr + vcol(k));
          else if constexpr (kRun == 2) *reinterpret_cast<float2*>(v) = *reinterpret_cast<const float2*>(vr + vcol(k));
          else v[0] = vr[vcol(k)];
#pragma unroll
          for (int e = 0; e < kRun; ++e) acc[k + e] = fmaf(w, v[e], acc[k + e]);
        }
    }
  }
  if (col >= ncol) return;
  if (a.splits > 1) {
    const size_t pc = ((static_cast<size_t>(b) * g.G + head) * a.splits + part) * ncol + col;
#pragma unroll
    for (int k = 0; k < kAcc; ++k)
      if (vcol(k) < a.dv) a.part_o[pc * a.dv + vcol(k)] = acc[k];
    if (lane == 0 && share == 0) {
      a.part_m[pc] = m;
      a.part_l[pc] = l;
    }
  } else {
    const size_t oc = (static_cast<size_t>(b) * a.Tq + qi) * a.H + head * hg + (cc - qi * hg);
    const float r = l == 0.f ? 0.f : 1.0f / l;
#pragma unroll
    for (int k = 0; k < kAcc; ++k)
      if (vcol(k) < a.dv) store_out(a.out, a.qdt, oc * a.dv + vcol(k), acc[k] * r);
    if (lane == 0 && share == 0 && a.lse != nullptr) a.lse[oc] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.693147180559945f;
  }
}

// out = sum_p 2^(m_p - m) o_p / sum_p 2^(m_p - m) l_p over a column's parts: a block for a
// column and 128 of its values.  The parts' weights come first (a thread a part), then each
// of the four warps sums every fourth part, four values a lane.
__global__ void __launch_bounds__(128) kv_attend_combine_kernel(const KvAttendArgs a, int slices) {
  __shared__ float wt[256];
  __shared__ float red[8];
  __shared__ float4 sums[4][32];
  pdl_wait();
  const KvGeom& g = a.g;
  const int hg = a.H / g.G, ncol = a.Tq * hg;
  const uint32_t cu = blockIdx.x / slices, slice = blockIdx.x - cu * slices;
  const uint32_t u = cu / ncol;
  const int col = static_cast<int>(cu - u * ncol);
  const int head = static_cast<int>(u % g.G), b = static_cast<int>(u / g.G);
  const size_t base = static_cast<size_t>(u) * a.splits * ncol + col;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float pm[2], pl[2];
  float m = -INFINITY;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int p = threadIdx.x + 128 * k;
    pl[k] = p < a.splits ? a.part_l[base + static_cast<size_t>(p) * ncol] : 0.f;
    pm[k] = p < a.splits ? a.part_m[base + static_cast<size_t>(p) * ncol] : 0.f;
    if (pl[k] != 0.f) m = fmaxf(m, pm[k]);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (lane == 0) red[warp] = m;
  __syncthreads();
  m = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
  float l = 0.f;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const float w = pl[k] != 0.f ? exp2f(pm[k] - m) : 0.f;
    wt[threadIdx.x + 128 * k] = w;
    l += pl[k] != 0.f ? w * pl[k] : 0.f;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  if (lane == 0) red[4 + warp] = l;
  __syncthreads();
  l = (red[4] + red[5]) + (red[6] + red[7]);
  const int qi = a.Tq == 1 ? 0 : col / hg;
  const size_t oc = (static_cast<size_t>(b) * a.Tq + qi) * a.H + head * hg + (col - qi * hg);
  const float r = l == 0.f ? 0.f : 1.0f / l;
  const float* po = a.part_o + base * a.dv;
  const size_t step = static_cast<size_t>(ncol) * a.dv;
  const int v = slice * 128 + lane * 4;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  if (a.dv % 4 == 0) {
    if (v < a.dv) {
#pragma unroll 8
      for (int p = warp; p < a.splits; p += 4) {
        const float4 f = *reinterpret_cast<const float4*>(po + p * step + v);
        const float w = wt[p];
        if (w != 0.f) {                                    // a part without tokens has stored nothing
          o.x = fmaf(w, f.x, o.x);
          o.y = fmaf(w, f.y, o.y);
          o.z = fmaf(w, f.z, o.z);
          o.w = fmaf(w, f.w, o.w);
        }
      }
    }
  } else {
    for (int p = warp; p < a.splits; p += 4) {
      const float w = wt[p];
      if (w == 0.f) continue;
      const float* f = po + p * step;
      if (v < a.dv) o.x = fmaf(w, f[v], o.x);
      if (v + 1 < a.dv) o.y = fmaf(w, f[v + 1], o.y);
      if (v + 2 < a.dv) o.z = fmaf(w, f[v + 2], o.z);
      if (v + 3 < a.dv) o.w = fmaf(w, f[v + 3], o.w);
    }
  }
  sums[warp][lane] = o;
  __syncthreads();
  if (warp == 0) {
    float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float4 f = sums[k][lane];
      s[0] += f.x;
      s[1] += f.y;
      s[2] += f.z;
      s[3] += f.w;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (v + e < a.dv) store_out(a.out, a.qdt, oc * a.dv + v + e, s[e] * r);
  }
  if (threadIdx.x == 0 && slice == 0 && a.lse != nullptr)
    a.lse[oc] = kv_lse(m, l);
}

size_t simt_smem(const KvAttendArgs& a, int team, int rows_used) {
  const int pitch = (rows_used + 31) / 32 * 32 + 4, dpad = (a.d + 3) & ~3;
  return static_cast<size_t>(kTile * pitch + kWarps / team * dpad + 2 * kWarps * kTile) * 4;
}

template <int kTeam>
int launch_team(const KvAttendArgs& a, cudaStream_t s) {
  const int ncol = a.Tq * (a.H / a.g.G), cols = kWarps / kTeam, col_blocks = (ncol + cols - 1) / cols;
  const int rows_used = (std::max(a.d, a.voff + a.dv) + 15) / 16 * 16;
  const size_t smem = simt_smem(a, kTeam, rows_used);
  const auto kern = a.voff % 4 == 0 && a.dv % 4 == 0 ? kv_attend_simt_kernel<true, kTeam> : kv_attend_simt_kernel<false, kTeam>;
  // the largest size, not this call's: two host threads may launch different ones
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
  if (e != cudaSuccess) return fail(LSA_ERR_CUDA, "kv_attend: %s", cudaGetErrorString(e));
  const long long grid = static_cast<long long>(a.g.B) * a.g.G * col_blocks * a.splits;
  kern<<<static_cast<unsigned>(grid), kWarps * 32, smem, s>>>(a, col_blocks, rows_used);
  return check_launch("kv_attend");
}

}  // namespace

void kv_attend_parts_simt(int B, int G, int ncol, long long max_tokens, int& team, int& splits) {
  const long long tiles = std::max<long long>(1, (max_tokens + kTile - 1) / kTile);
  // Parts of two tiles: 4096 tokens of 576 codes under 8 fp32 columns take 16.5 us (33 with parts of
  // eight, 18 with one), 4 x 2048 listed tokens 21 (38, 23).
  const long long parts = (tiles + 1) / 2;
  auto units = [&](int t) { return static_cast<long long>(B) * G * ((ncol + kWarps / t - 1) / (kWarps / t)); };
  // A block of fewer columns reads the same rows, so a team takes more than one warp where warps
  // would have no column, and where there are fewer blocks than SMs.
  team = 1;
  while (team < kWarps && (units(2 * team) == units(team) || units(2 * team) * parts <= 148)) team *= 2;
  splits = static_cast<int>(std::max<long long>(1, std::min<long long>({(4 * 148 + units(team) - 1) / units(team), parts, 256})));
}

int launch_kv_attend_simt(const KvAttendArgs& a, int team, cudaStream_t s) {
  switch (team) {
    case 1: return launch_team<1>(a, s);
    case 2: return launch_team<2>(a, s);
    case 4: return launch_team<4>(a, s);
    default: return launch_team<8>(a, s);
  }
}

int launch_kv_attend_combine(const KvAttendArgs& a, cudaStream_t s) {
  const int slices = (a.dv + 127) / 128;
  const long long grid = static_cast<long long>(a.g.B) * a.g.G * a.Tq * (a.H / a.g.G) * slices;   // at most 2^26
  const cudaError_t e = launch_dependent(kv_attend_combine_kernel, dim3(static_cast<unsigned>(grid)), dim3(128), 0, s, a, slices);
  if (e != cudaSuccess) return fail(LSA_ERR_CUDA, "kv_attend: %s", cudaGetErrorString(e));
  return check_launch("kv_attend_combine");
}

}  // namespace lsa
