// Root-mean-square norm with the residual's addition, bf16 and / or e4m3 out.
//
//   s = x + r,  n = s / sqrt(mean(s^2) + eps) * w,  r' = bf16(s),  y = bf16(n),
//   code = e4m3(n / scale),  scale = max|n| / 448 over a run of columns.
//
// One pass over memory: a team of threads holds its row's s in registers
// between the sum of squares and the scaling, so every input is read once and
// every output written once (8 to 9 bytes an element with the residual and
// the codes); the kernel is bound by HBM: 52 us in a chain of calls, 58 from cold
// caches, for 8191 rows of 4096 with the residual, bf16 and codes (303 MB, 5.8 and
// 5.2 TB/s; a plain copy of as many bytes from cold caches takes 54).  The sums
// and n stay in fp32 and each output is rounded once; the norm uses s before its
// rounding to bf16.
#include <cuda_fp8.h>

#include "fl_common.cuh"

using namespace fl;

namespace {

struct NormParams {
  const __nv_bfloat16* x;
  const __nv_bfloat16* r;
  const __nv_bfloat16* w;
  __nv_bfloat16* y;
  __nv_bfloat16* ro;
  uint8_t* codes;
  float* scales;
  int64_t xs, rs, ys, ros;
  long long rows;
  int heads, H, group;
  float eps;
};

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// 8 elements from column c on; those at or past H read as 0.
template <bool VEC>
__device__ __forceinline__ void load8(const __nv_bfloat16* row, int c, int H, float (&v)[8]) {
  if constexpr (VEC) {
    uint4 u = make_uint4(0, 0, 0, 0);
    if (c < H) u = *reinterpret_cast<const uint4*>(row + c);
    const uint32_t a[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(a[i] << 16);
      v[2 * i + 1] = __uint_as_float(a[i] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = c + i < H ? __bfloat162float(row[c + i]) : 0.f;
  }
}

template <bool VEC>
__device__ __forceinline__ void store8(__nv_bfloat16* row, int c, int H, const float (&v)[8]) {
  if constexpr (VEC) {
    if (c < H)
      *reinterpret_cast<uint4*>(row + c) =
          make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < H) row[c + i] = __float2bfloat16_rn(v[i]);
  }
}

// Sum or maximum over the team of TPR threads (a warp, or the whole CTA).
template <int TPR, bool MAX>
__device__ __forceinline__ float team_reduce(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float u = __shfl_xor_sync(0xffffffffu, v, o);
    v = MAX ? fmaxf(v, u) : v + u;
  }
  if constexpr (TPR > 32) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) red[warp] = v;
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int i = 1; i < TPR / 32; ++i) v = MAX ? fmaxf(v, red[i]) : v + red[i];
  }
  return v;
}

// A row whose mean square is not among these, for which its squares are summed
// once more with the values times a power of two: above, fp32 has no number for
// the sum (values beyond 1e19 / sqrt(H), infinities, NaN); below, with next to no
// eps, the squares are rounded to its last numbers or to 0.
constexpr float kMeanMin = 7.888609052210118e-31f, kMeanMax = 3.4028234663852886e38f;   // 2^-100, the largest
__device__ __forceinline__ bool odd_mean(float ms) { return !(ms >= kMeanMin && ms <= kMeanMax); }
// 2^90 or 2^-72: the squares of all fp32 numbers that can lead here, and their sum, are normal numbers.
__device__ __forceinline__ float odd_factor(float ms) { return ms < 1.f ? 1.2379400392853803e27f : 2.117582368135751e-22f; }
// 1 / sqrt(mean + eps) from the sum with the values times f, and what the
// values have to be multiplied by before (x: tiny values' reciprocal may pass
// fp32).  A row with an infinity or a NaN: NaN.
__device__ __forceinline__ float2 odd_rstd(float sum, float f, int H, float eps) {
  const float ms = sum / static_cast<float>(H) + eps * f * f, r = rsqrtf(ms);
  return f > 1.f ? make_float2(f, r) : make_float2(1.f, ms <= kMeanMax ? r * f : __int_as_float(0x7fffffff));
}

// TPR threads hold one row, V vectors of 8 columns each: thread i has the
// vectors i, i + TPR, ...  A CTA is one team, or four when a team is a warp.
// V is what the row needs: 8191 rows of 5120 columns take 33 us with 3 vectors a
// thread and 40 with 4, 16000 rows of 2048 22.5 with 2 and 25 with 4.
// Teams of 128 are held to 64 registers, for 8 of them on an SM (rows of 4096
// with residual and codes: 56 us; 7 of them 64, 9 of them, which spill, 66).
template <int TPR, int V, bool VEC>
__global__ void __launch_bounds__(TPR == 32 ? 128 : TPR, TPR == 128 ? 8 : 1) k_rmsnorm(const NormParams p) {
  __shared__ float red[3][TPR / 32];
  pdl_launch_dependents();
  pdl_wait();
  constexpr int kTeams = TPR == 32 ? 4 : 1;
  const int t = threadIdx.x % TPR;
  const long long row = static_cast<long long>(blockIdx.x) * kTeams + threadIdx.x / TPR;
  if (row >= p.rows) return;   // a whole team at once
  const long long m = row / p.heads;
  const int64_t off = (row - m * p.heads) * p.H;
  const __nv_bfloat16* x = p.x + m * p.xs + off;
  float s[V][8];
#pragma unroll
  for (int i = 0; i < V; ++i) load8<VEC>(x, (i * TPR + t) * 8, p.H, s[i]);
  if (p.r) {
    const __nv_bfloat16* r = p.r + m * p.rs + off;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float u[8];
      load8<VEC>(r, (i * TPR + t) * 8, p.H, u);
#pragma unroll
      for (int j = 0; j < 8; ++j) s[i][j] += u[j];
    }
  }
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) sum = fmaf(s[i][j], s[i][j], sum);
  sum = team_reduce<TPR, false>(sum, red[0]);
  const float ms = sum / static_cast<float>(p.H) + p.eps;
  float rstd = rsqrtf(ms);
  if (p.ro) {
    __nv_bfloat16* ro = p.ro + m * p.ros + off;
#pragma unroll
    for (int i = 0; i < V; ++i) store8<VEC>(ro, (i * TPR + t) * 8, p.H, s[i]);
  }
  if (odd_mean(ms)) {   // (the same in the whole team)
    const float f = odd_factor(ms);
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) sum = fmaf(s[i][j] * f, s[i][j] * f, sum);
    const float2 by = odd_rstd(team_reduce<TPR, false>(sum, red[2]), f, p.H, p.eps);
    rstd = by.y;
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) s[i][j] *= by.x;
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    float w[8];
    if (p.w) {
      load8<VEC>(p.w, (i * TPR + t) * 8, p.H, w);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = 1.f;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) s[i][j] = s[i][j] * rstd * w[j];
  }
  if (p.y) {
    __nv_bfloat16* y = p.y + m * p.ys + off;
#pragma unroll
    for (int i = 0; i < V; ++i) store8<VEC>(y, (i * TPR + t) * 8, p.H, s[i]);
  }
  if (p.codes) {
    float top[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      top[i] = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) top[i] = fmaxf(top[i], fabsf(s[i][j]));
    }
    if (p.group) {
      // a run of `group` columns is group / 8 neighbouring lanes
      for (int o = 1; o < p.group / 8; o <<= 1)
#pragma unroll
        for (int i = 0; i < V; ++i) top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], o));
    } else {
#pragma unroll
      for (int i = 1; i < V; ++i) top[0] = fmaxf(top[0], top[i]);
      const float a = team_reduce<TPR, true>(top[0], red[1]);
#pragma unroll
      for (int i = 0; i < V; ++i) top[i] = a;
    }
    // 1 / scale of a scale below fp32's normal numbers may be infinite: such a run
    // and its scale are taken times 2^64.
    constexpr float kTiny = 448.f * 1.1754943508222875e-38f, kLift = 18446744073709551616.f;
    bool tiny = false;
#pragma unroll
    for (int i = 0; i < V; ++i) tiny |= top[i] < kTiny;
    if (tiny) {
#pragma unroll
      for (int i = 0; i < V; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) s[i][j] *= top[i] < kTiny ? kLift : 1.f;
    }
    const int ng = p.group ? p.H / p.group : 1;
    uint8_t* cr = p.codes + row * p.H;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (i * TPR + t) * 8;
      if (c >= p.H) continue;
      const float scale = __fdiv_rn(top[i], 448.f);
      const float up = top[i] < kTiny ? scale * kLift : scale;
      const float inv = scale > 0.f ? __frcp_rn(up) : 0.f;   // (n times it: n / scale within 2^-23)
      if (p.group ? c % p.group == 0 : c == 0) p.scales[row * ng + (p.group ? c / p.group : 0)] = scale;
      uint32_t o[2] = {0, 0};
#pragma unroll
      for (int j = 0; j < 8; j += 2) {   // (adding 0: a run of zeros has codes 0 whatever their signs; NaN stays)
        const float2 v = make_float2(fmaf(s[i][j], inv, 0.f), fmaf(s[i][j + 1], inv, 0.f));
        o[j >> 2] |= static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(v, __NV_SATFINITE, __NV_E4M3)) << (8 * (j & 3));
      }
      if constexpr (VEC) {
        *reinterpret_cast<uint2*>(cr + c) = make_uint2(o[0], o[1]);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (c + j < p.H) cr[c + j] = static_cast<uint8_t>(o[j >> 2] >> (8 * (j & 3)));
      }
    }
  }
}

// The rows of a warp of the kernel below, once one of them has an odd mean: all
// from the start, in a function of its own, so that the kernel's common path
// keeps its registers (heads of 128: 26.2 us, as a branch in it 27.9).
template <int LPR>
__device__ __noinline__ void odd_narrow(const NormParams& p, unsigned row) {
  const unsigned m = row / static_cast<unsigned>(p.heads);
  const int c = threadIdx.x % LPR * 8, H = row < p.rows ? p.H : 0;
  const int off = static_cast<int>(row - m * p.heads) * p.H;
  float s[8], w[8];
  load8<true>(p.x + (H ? m * p.xs + off : 0), c, H, s);
  if (p.r) {
    load8<true>(p.r + (H ? m * p.rs + off : 0), c, H, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) s[j] += w[j];
  }
  float f = 1.f;   // for an ordinary row
  float2 rstd;
  for (int pass = 0; pass < 2; ++pass) {
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) sum = fmaf(s[j] * f, s[j] * f, sum);
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const float ms = sum / static_cast<float>(p.H) + p.eps;
    if (pass == 1) {
      if (f != 1.f) rstd = odd_rstd(sum, f, p.H, p.eps);
    } else {
      rstd = make_float2(1.f, rsqrtf(ms));
      if (odd_mean(ms)) f = odd_factor(ms);
    }
  }
  if (!H) return;
  if (p.ro) store8<true>(p.ro + m * p.ros + off, c, H, s);
  if (p.w) load8<true>(p.w, c, H, w);
#pragma unroll
  for (int j = 0; j < 8; ++j) s[j] = s[j] * rstd.x * rstd.y * (p.w ? w[j] : 1.f);
  store8<true>(p.y + m * p.ys + off, c, H, s);
}

// Rows of at most 8 LPR columns (heads of 64 or 128) without codes: LPR lanes
// hold one, a vector each.  (8191 tokens of 32 heads of 128, 134 MB: 26 us, 5.2
// TB/s; a warp a row as above, half of it idle, 68 us; before rows of odd means had
// their path, two rows a team took 24 and four 25.)
constexpr int kNarrowThreads = 256;
template <int LPR>
__global__ void __launch_bounds__(kNarrowThreads, 8) k_rmsnorm_narrow(const __grid_constant__ NormParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const unsigned row = blockIdx.x * (kNarrowThreads / LPR) + threadIdx.x / LPR;
  const unsigned m = row / static_cast<unsigned>(p.heads);
  const int c = threadIdx.x % LPR * 8;
  const int off = static_cast<int>(row - m * p.heads) * p.H;
  const int H = row < p.rows ? p.H : 0;   // (past the last row: zeros, for the shuffles)
  float s[8], w[8];
  load8<true>(p.x + (H ? m * p.xs + off : 0), c, H, s);
  if (p.r) {
    float u[8];
    load8<true>(p.r + (H ? m * p.rs + off : 0), c, H, u);
#pragma unroll
    for (int j = 0; j < 8; ++j) s[j] += u[j];
  }
  if (p.w) {
    load8<true>(p.w, c, H, w);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = 1.f;
  }
  float sum = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) sum = fmaf(s[j], s[j], sum);
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  const float ms = sum / static_cast<float>(p.H) + p.eps;
  if (__any_sync(0xffffffffu, odd_mean(ms))) {
    odd_narrow<LPR>(p, row);   // (nothing of the warp's rows has been stored)
    return;
  }
  const float rstd = rsqrtf(ms);
  if (!H) return;
  if (p.ro) store8<true>(p.ro + m * p.ros + off, c, H, s);
#pragma unroll
  for (int j = 0; j < 8; ++j) s[j] = s[j] * rstd * w[j];
  store8<true>(p.y + m * p.ys + off, c, H, s);
}

template <int LPR>
int launch_narrow(const NormParams& p, cudaStream_t s) {
  constexpr int kRows = kNarrowThreads / LPR;
  return flh::launch_early(k_rmsnorm_narrow<LPR>, dim3(static_cast<unsigned>((p.rows + kRows - 1) / kRows)),
                           dim3(kNarrowThreads), 0, s, p);
}

template <int TPR, int V>
int launch_norm(const NormParams& p, bool vec, cudaStream_t s) {
  constexpr int kTeams = TPR == 32 ? 4 : 1;
  const long long grid = (p.rows + kTeams - 1) / kTeams;
  if (grid > 0x7fffffffll) return FL_ERR_UNSUPPORTED;
  const dim3 g(static_cast<unsigned>(grid)), b(TPR == 32 ? 128 : TPR);
  return vec ? flh::launch_early(k_rmsnorm<TPR, V, true>, g, b, 0, s, p) : flh::launch_early(k_rmsnorm<TPR, V, false>, g, b, 0, s, p);
}

// Teams grow before they would need more than 4 vectors a thread, so one vector
// happens in teams of 32 only, two in teams of 32 and 128.
template <int V>
int pick_team(const NormParams& p, int tpr, bool vec, cudaStream_t s) {
  if constexpr (V >= 2) {
    if (tpr == 128) return launch_norm<128, V>(p, vec, s);
  }
  if constexpr (V >= 3) {
    if (tpr == 256) return launch_norm<256, V>(p, vec, s);
    if (tpr == 512) return launch_norm<512, V>(p, vec, s);
    if (tpr == 1024) return launch_norm<1024, V>(p, vec, s);
  }
  return launch_norm<32, V>(p, vec, s);
}

bool aligned_to(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace

extern "C" int fl_rmsnorm(const void* x, int64_t x_stride, const void* residual, int64_t residual_stride,
                          const void* weight, float eps, int M, int heads, int H, void* y, int64_t y_stride,
                          void* residual_out, int64_t residual_out_stride, void* codes, float* scales, int group,
                          fl_stream_t stream) {
  if (!x || (!y && !codes) || (y && y == residual_out) || (codes != nullptr) != (scales != nullptr)) return FL_ERR_ARG;
  if (M < 1 || heads < 1 || H < 1 || !(eps >= 0.f) || eps > 3.0e38f) return FL_ERR_ARG;
  if (H > 32768) return FL_ERR_UNSUPPORTED;
  if (group != 0 && group != 64 && group != 128 && group != 256) return FL_ERR_UNSUPPORTED;
  if (!codes && group) return FL_ERR_ARG;
  if (group && H % group) return FL_ERR_ARG;
  const int64_t w = static_cast<int64_t>(heads) * H;
  if (x_stride < w || (residual && residual_stride < w) || (y && y_stride < w) ||
      (residual_out && residual_out_stride < w))
    return FL_ERR_ARG;
  const void* ptr[5] = {x, residual, weight, y, residual_out};
  const int64_t st[5] = {x_stride, residual ? residual_stride : 0, 0, y ? y_stride : 0,
                         residual_out ? residual_out_stride : 0};
  bool vec = H % 8 == 0 && aligned_to(codes, 8);
  for (int i = 0; i < 5; ++i) {
    if (!aligned_to(ptr[i], 2)) return FL_ERR_ARG;
    vec = vec && aligned_to(ptr[i], 16) && st[i] % 8 == 0;
  }
  if (!aligned_to(scales, 4)) return FL_ERR_ARG;
  NormParams p;
  p.x = static_cast<const __nv_bfloat16*>(x);
  p.r = static_cast<const __nv_bfloat16*>(residual);
  p.w = static_cast<const __nv_bfloat16*>(weight);
  p.y = static_cast<__nv_bfloat16*>(y);
  p.ro = static_cast<__nv_bfloat16*>(residual_out);
  p.codes = static_cast<uint8_t*>(codes);
  p.scales = scales;
  p.xs = x_stride, p.rs = residual_stride, p.ys = y_stride, p.ros = residual_out_stride;
  p.rows = static_cast<long long>(M) * heads;
  p.heads = heads, p.H = H, p.group = group, p.eps = eps;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (vec && !codes && H <= 128 && w < (1ll << 31) && p.rows < 0x7fffffffll) return H <= 64 ? launch_narrow<8>(p, s) : launch_narrow<16>(p, s);
  int tpr = 32;
  while (tpr < 1024 && tpr * 32 < H) tpr = tpr == 32 ? 128 : 2 * tpr;   // at most 4 vectors a thread
  if (tpr * 8 >= H) return pick_team<1>(p, tpr, vec, s);
  if (tpr * 16 >= H) return pick_team<2>(p, tpr, vec, s);
  if (tpr * 24 >= H) return pick_team<3>(p, tpr, vec, s);
  return pick_team<4>(p, tpr, vec, s);
}
