// Rotary positions with several axes for queries and keys in one launch.
//
// Pair i = (u, v) of every head of token t turns by a = pos[axis(i)][t] * f_i:
//   u' = u cos a - v sin a,  v' = v cos a + u sin a.
// The angle is held in turns, in 64-bit fixed point: step_i = frac(f_i / 2 pi)
// * 2^64 and pos * step_i mod 2^64 is the angle's fraction of a turn, exact
// but for the rounding of step_i (2^-53 of f_i; at position 2^20 that is
// 2^-33 of a turn), with no table and no fp64 in the loop.  Its top 32 bits go
// through sincospif.  The sines of one token's pairs are computed once, into
// shared memory, for all of its heads, so the kernel is bound by HBM: 4 bytes
// an element.
#include "fl_common.cuh"

using namespace fl;

namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopePairs = 512;    // most pairs of a head (D <= 1024)
constexpr int kRopeTable = 1024;   // sines held at once: tokens of a pass x pairs

struct RopeParams {
  const __nv_bfloat16* q;
  const __nv_bfloat16* k;
  __nv_bfloat16* qo;
  __nv_bfloat16* ko;
  const int32_t* pos;
  const double* freq;
  int64_t qs, ks, qos, kos;
  int T, Hq, Hk, D, rot, style, axes, tt;   // tt: tokens of a pass
  int end[FL_ROPE_MAX_AXES];                // first pair past each axis's section
};

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float lo_f(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float hi_f(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }

template <bool VEC>
__global__ void __launch_bounds__(kRopeThreads) k_rope(const RopeParams p) {
  __shared__ unsigned long long step[kRopePairs];
  __shared__ __align__(16) float2 sc[kRopeTable];   // (cos, sin)
  const int pairs = p.rot / 2, heads = p.Hq + p.Hk;
  for (int i = threadIdx.x; i < pairs; i += kRopeThreads) {
    const double turns = p.freq[i] * 0.15915494309189533576888376337251436;   // 1 / (2 pi)
    step[i] = __double2ull_rn((turns - floor(turns)) * 18446744073709551616.0);
  }
  // units of work of a head: 8 elements of either half (halves) or 8 adjacent
  // elements (pairs), or one pair or one copied element
  const int turn_units = VEC ? (p.style == FL_ROPE_HALVES ? pairs / 8 : p.rot / 8) : pairs;
  const int units = turn_units + (VEC ? (p.D - p.rot) / 8 : p.D - p.rot);
  for (int t0 = blockIdx.x * p.tt; t0 < p.T; t0 += gridDim.x * p.tt) {
    const int nt = min(p.tt, p.T - t0);
    __syncthreads();
    for (int i = threadIdx.x; i < nt * pairs; i += kRopeThreads) {
      const int t = i / pairs, pr = i - t * pairs;
      int a = 0;
      while (a + 1 < p.axes && pr >= p.end[a]) ++a;
      const long long at = p.pos[static_cast<int64_t>(a) * p.T + t0 + t];
      const unsigned long long ph = static_cast<unsigned long long>(at) * step[pr];
      const float half_turns = static_cast<float>(static_cast<int32_t>(ph >> 32)) * 4.656612873077392578125e-10f;
      float s, c;
      sincospif(half_turns, &s, &c);
      sc[i] = make_float2(c, s);
    }
    __syncthreads();
    const int n = nt * heads * units;
    for (int i = threadIdx.x; i < n; i += kRopeThreads) {
      const int hh = i / units, u = i - hh * units;
      const int t = hh / heads, h = hh - t * heads;
      const int64_t tok = t0 + t;
      const __nv_bfloat16* src = h < p.Hq ? p.q + tok * p.qs + h * p.D : p.k + tok * p.ks + (h - p.Hq) * p.D;
      __nv_bfloat16* dst = h < p.Hq ? p.qo + tok * p.qos + h * p.D : p.ko + tok * p.kos + (h - p.Hq) * p.D;
      const float2* cs = sc + t * pairs;
      if (u >= turn_units) {   // past the rotated part
        const int c = p.rot + (u - turn_units) * (VEC ? 8 : 1);
        if constexpr (VEC)
          *reinterpret_cast<uint4*>(dst + c) = *reinterpret_cast<const uint4*>(src + c);
        else
          dst[c] = src[c];
      } else if constexpr (!VEC) {
        const int a = p.style == FL_ROPE_HALVES ? u : 2 * u, b = p.style == FL_ROPE_HALVES ? u + pairs : 2 * u + 1;
        const float x = __bfloat162float(src[a]), y = __bfloat162float(src[b]);
        dst[a] = __float2bfloat16_rn(x * cs[u].x - y * cs[u].y);
        dst[b] = __float2bfloat16_rn(y * cs[u].x + x * cs[u].y);
      } else if (p.style == FL_ROPE_HALVES) {
        const uint4 xv = *reinterpret_cast<const uint4*>(src + 8 * u);
        const uint4 yv = *reinterpret_cast<const uint4*>(src + pairs + 8 * u);
        const uint32_t xa[4] = {xv.x, xv.y, xv.z, xv.w}, ya[4] = {yv.x, yv.y, yv.z, yv.w};
        uint32_t xo[4], yo[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float4 w = *reinterpret_cast<const float4*>(cs + 8 * u + 2 * j);
          const float x0 = lo_f(xa[j]), x1 = hi_f(xa[j]), y0 = lo_f(ya[j]), y1 = hi_f(ya[j]);
          xo[j] = pack_bf16(x0 * w.x - y0 * w.y, x1 * w.z - y1 * w.w);
          yo[j] = pack_bf16(y0 * w.x + x0 * w.y, y1 * w.z + x1 * w.w);
        }
        *reinterpret_cast<uint4*>(dst + 8 * u) = make_uint4(xo[0], xo[1], xo[2], xo[3]);
        *reinterpret_cast<uint4*>(dst + pairs + 8 * u) = make_uint4(yo[0], yo[1], yo[2], yo[3]);
      } else {
        const uint4 xv = *reinterpret_cast<const uint4*>(src + 8 * u);
        const uint32_t xa[4] = {xv.x, xv.y, xv.z, xv.w};
        uint32_t xo[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 w = cs[4 * u + j];
          const float x = lo_f(xa[j]), y = hi_f(xa[j]);
          xo[j] = pack_bf16(x * w.x - y * w.y, y * w.x + x * w.y);
        }
        *reinterpret_cast<uint4*>(dst + 8 * u) = make_uint4(xo[0], xo[1], xo[2], xo[3]);
      }
    }
  }
}

bool aligned_to(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace

extern "C" int fl_rope(const void* q, int64_t q_stride, int Hq, const void* k, int64_t k_stride, int Hk, int T, int D,
                       int rot, int style, const int32_t* positions, int n_axes, const int32_t* sections,
                       const double* inv_freq, void* q_out, int64_t q_out_stride, void* k_out, int64_t k_out_stride,
                       fl_stream_t stream) {
  if (!q || !q_out || !positions || !inv_freq || (Hk > 0 && (!k || !k_out))) return FL_ERR_ARG;
  if (T < 1 || Hq < 1 || Hk < 0 || D < 2 || rot < 2 || rot > D || rot % 2) return FL_ERR_ARG;
  if (D > 1024 || static_cast<int64_t>(Hq) + Hk > 65536) return FL_ERR_UNSUPPORTED;
  if (style != FL_ROPE_HALVES && style != FL_ROPE_PAIRS) return FL_ERR_ARG;
  if (n_axes < 1 || n_axes > FL_ROPE_MAX_AXES || (n_axes > 1 && !sections)) return FL_ERR_ARG;
  const int64_t wq = static_cast<int64_t>(Hq) * D, wk = static_cast<int64_t>(Hk) * D;
  if (q_stride < wq || q_out_stride < wq || (Hk > 0 && (k_stride < wk || k_out_stride < wk))) return FL_ERR_ARG;
  if (!aligned_to(q, 2) || !aligned_to(k, 2) || !aligned_to(q_out, 2) || !aligned_to(k_out, 2) ||
      !aligned_to(positions, 4) || !aligned_to(inv_freq, 8))
    return FL_ERR_ARG;
  RopeParams p;
  int sum = 0;
  for (int a = 0; a < FL_ROPE_MAX_AXES; ++a) {
    const int n = a >= n_axes ? 0 : sections ? sections[a] : rot / 2;
    if (n < 0 || n > rot / 2) return FL_ERR_ARG;
    sum += n;
    p.end[a] = sum;
  }
  if (sum != rot / 2) return FL_ERR_ARG;
  p.q = static_cast<const __nv_bfloat16*>(q), p.k = static_cast<const __nv_bfloat16*>(k);
  p.qo = static_cast<__nv_bfloat16*>(q_out), p.ko = static_cast<__nv_bfloat16*>(k_out);
  p.pos = positions, p.freq = inv_freq;
  p.qs = q_stride, p.ks = k_stride, p.qos = q_out_stride, p.kos = k_out_stride;
  p.T = T, p.Hq = Hq, p.Hk = Hk, p.D = D, p.rot = rot, p.style = style, p.axes = n_axes;
  const int pairs = rot / 2;
  bool vec = D % 8 == 0 && pairs % 8 == 0 && aligned_to(q, 16) && aligned_to(q_out, 16) && q_stride % 8 == 0 &&
             q_out_stride % 8 == 0;
  if (Hk > 0)
    vec = vec && aligned_to(k, 16) && aligned_to(k_out, 16) && k_stride % 8 == 0 && k_out_stride % 8 == 0;
  // tokens of a pass: as many as give every thread of a CTA a unit, within the table
  const int per = (Hq + Hk) * (vec ? (style == FL_ROPE_HALVES ? D / 16 : D / 8) : pairs);
  int tt = kRopeThreads / (per > 0 ? per : 1);
  if (tt > kRopeTable / pairs) tt = kRopeTable / pairs;
  if (tt < 1) tt = 1;
  p.tt = tt;
  const int64_t passes = (static_cast<int64_t>(T) + tt - 1) / tt;
  const int64_t most = 8ll * flh::sm_count();   // resident CTAs: 8 of 256 threads on an SM
  const unsigned grid = static_cast<unsigned>(passes < most ? passes : most);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (vec)
    k_rope<true><<<grid, kRopeThreads, 0, s>>>(p);
  else
    k_rope<false><<<grid, kRopeThreads, 0, s>>>(p);
  return cudaGetLastError() == cudaSuccess ? FL_OK : FL_ERR_CUDA;
}
