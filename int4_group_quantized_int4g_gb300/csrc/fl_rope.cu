// Rotary positions with several axes for queries and keys in one launch.
//
// Pair i = (u, v) of every head of token t turns by a = pos[axis(i)][t] * f_i:
//   u' = u cos a - v sin a,  v' = v cos a + u sin a.
// The angle is held in turns, in 64-bit fixed point: step_i = frac(f_i / 2 pi)
// * 2^64 and pos * step_i mod 2^64 is the angle's fraction of a turn, exact
// but for the rounding of step_i (2^-53 of f_i; at position 2^20 that is
// 2^-33 of a turn), with no table and no fp64 in the loop.  Its top 32 bits go
// through sincospif.  The sines of a token's pairs are computed once, into
// shared memory, for all of its heads, in the order in which neighbouring
// threads read them (pair by pair they met four-way bank conflicts: 64 us for
// 16381 tokens of 36 heads of 128 instead of 54).  Bound by HBM, 4 bytes an
// element: 302 MB there, 5.6 TB/s, what a plain copy reaches.
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
  int end0, end1, end2;                     // first pair past the first, second, third axis's section
};

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float lo_f(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float hi_f(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }

// What one thread moves: 8 pairs of either half (halves), 4 pairs (pairs), 8
// copied elements; or, element by element, one pair or one copied element.
template <bool VEC>
struct Unit {
  uint4 a, b;
  const __nv_bfloat16* src;
  __nv_bfloat16* dst;
  int tok;
};

template <bool VEC>
__global__ void __launch_bounds__(kRopeThreads, 5) k_rope(const RopeParams p) {
  __shared__ unsigned long long step[kRopePairs];
  __shared__ __align__(16) float2 sc[kRopeTable];   // (cos, sin)
  pdl_launch_dependents();
  pdl_wait();
  const int pairs = p.rot / 2, heads = p.Hq + p.Hk;
  const bool halves = p.style == FL_ROPE_HALVES;
  const int turned = VEC ? (halves ? pairs / 8 : p.rot / 8) : pairs;   // units of a head that turn
  const int units = turned + (VEC ? (p.D - p.rot) / 8 : p.D - p.rot);
  // A thread keeps its unit of a head and steps through the heads of the CTA's
  // tokens; `lanes` threads have a head, `step_h` heads go at a time.
  const int lanes = min(units, kRopeThreads), step_h = kRopeThreads / lanes;
  const int h0 = threadIdx.x / lanes;
  const int t0 = blockIdx.x * p.tt, nt = min(p.tt, p.T - t0);
  int u = threadIdx.x - h0 * lanes;
  int at = 0, t = 0, h = 0, left = 0;   // the unit's first element, the next head, heads left
  auto begin = [&]() {
    at = u < turned ? (VEC ? 8 * u : 0) : p.rot + (u - turned) * (VEC ? 8 : 1);
    t = h0 / heads, h = h0 - t * heads;
    left = h0 < step_h ? (nt * heads - h0 + step_h - 1) / step_h : 0;
  };
  auto load = [&](Unit<VEC>& x) {   // of the thread's next head
    x.tok = t;
    const int64_t tok = t0 + t;
    x.src = h < p.Hq ? p.q + tok * p.qs + h * p.D : p.k + tok * p.ks + (h - p.Hq) * p.D;
    x.dst = h < p.Hq ? p.qo + tok * p.qos + h * p.D : p.ko + tok * p.kos + (h - p.Hq) * p.D;
    if constexpr (VEC) {
      x.a = *reinterpret_cast<const uint4*>(x.src + at);
      if (u < turned && halves) x.b = *reinterpret_cast<const uint4*>(x.src + pairs + at);
    }
    h += step_h;
    while (h >= heads) h -= heads, ++t;
  };
  // the first loads go out before the sines are computed
  Unit<VEC> x, y;
  begin();
  if (left > 0) load(x);
  if (left > 1) load(y);

  for (int i = threadIdx.x; i < pairs; i += kRopeThreads) {
    const double turns = p.freq[i] * 0.15915494309189533576888376337251436;   // 1 / (2 pi)
    step[i] = __double2ull_rn((turns - floor(turns)) * 18446744073709551616.0);
  }
  __syncthreads();
  // Where a token's pair lies: the unit's pairs two by two, all units' first two,
  // then their next, so that neighbouring lanes read neighbouring 16 bytes.
  auto place = [&](int pr) {
    if (!VEC) return pr;
    const int per = halves ? 8 : 4, unit = pr / per, k = pr - unit * per;
    return ((k >> 1) * turned + unit) * 2 + (k & 1);
  };
  for (int i = threadIdx.x; i < nt * pairs; i += kRopeThreads) {
    const int tok = i / pairs, pr = i - tok * pairs;
    const int a = (pr >= p.end0) + (pr >= p.end1) + (pr >= p.end2);
    const long long pos = p.pos[static_cast<int64_t>(a) * p.T + t0 + tok];
    const unsigned long long ph = static_cast<unsigned long long>(pos) * step[pr];
    const float half_turns = static_cast<float>(static_cast<int32_t>(ph >> 32)) * 4.656612873077392578125e-10f;
    float sn, c;
    sincospif(half_turns, &sn, &c);
    sc[tok * pairs + place(pr)] = make_float2(c, sn);
  }
  __syncthreads();
  {
    auto store = [&](const Unit<VEC>& x) {
      const float2* cs = sc + x.tok * pairs;
      if constexpr (!VEC) {
        if (u >= turned) {
          x.dst[at] = x.src[at];
        } else {
          const int a = halves ? u : 2 * u, b = halves ? u + pairs : 2 * u + 1;
          const float v = __bfloat162float(x.src[a]), w = __bfloat162float(x.src[b]);
          x.dst[a] = __float2bfloat16_rn(v * cs[u].x - w * cs[u].y);
          x.dst[b] = __float2bfloat16_rn(w * cs[u].x + v * cs[u].y);
        }
      } else if (u >= turned) {   // past the rotated part
        *reinterpret_cast<uint4*>(x.dst + at) = x.a;
      } else if (halves) {
        const uint32_t xa[4] = {x.a.x, x.a.y, x.a.z, x.a.w}, ya[4] = {x.b.x, x.b.y, x.b.z, x.b.w};
        uint32_t xo[4], yo[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float4 w = *reinterpret_cast<const float4*>(cs + (j * turned + u) * 2);
          const float x0 = lo_f(xa[j]), x1 = hi_f(xa[j]), y0 = lo_f(ya[j]), y1 = hi_f(ya[j]);
          xo[j] = pack_bf16(x0 * w.x - y0 * w.y, x1 * w.z - y1 * w.w);
          yo[j] = pack_bf16(y0 * w.x + x0 * w.y, y1 * w.z + x1 * w.w);
        }
        *reinterpret_cast<uint4*>(x.dst + at) = make_uint4(xo[0], xo[1], xo[2], xo[3]);
        *reinterpret_cast<uint4*>(x.dst + pairs + at) = make_uint4(yo[0], yo[1], yo[2], yo[3]);
      } else {
        const uint32_t xa[4] = {x.a.x, x.a.y, x.a.z, x.a.w};
        uint32_t xo[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 w = cs[((j >> 1) * turned + u) * 2 + (j & 1)];
          const float v = lo_f(xa[j]), z = hi_f(xa[j]);
          xo[j] = pack_bf16(v * w.x - z * w.y, z * w.x + v * w.y);
        }
        *reinterpret_cast<uint4*>(x.dst + at) = make_uint4(xo[0], xo[1], xo[2], xo[3]);
      }
    };
    for (;;) {
      while (left > 0) {   // two heads at a time
        store(x);
        if (left > 1) store(y);
        left -= 2;
        if (left > 0) load(x);
        if (left > 1) load(y);
      }
      u += lanes;   // (a head of more units than the CTA has threads)
      if (u >= units || h0 >= step_h) break;
      begin();
      if (left > 0) load(x);
      if (left > 1) load(y);
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
  int sum = 0, end[FL_ROPE_MAX_AXES];
  for (int a = 0; a < FL_ROPE_MAX_AXES; ++a) {
    const int n = a >= n_axes ? 0 : sections ? sections[a] : rot / 2;
    if (n < 0 || n > rot / 2) return FL_ERR_ARG;
    sum += n;
    end[a] = sum;
  }
  if (sum != rot / 2) return FL_ERR_ARG;
  p.end0 = end[0], p.end1 = end[1], p.end2 = end[2];
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
  // Tokens of a CTA: as many as fit the table, up to 8, but with few tokens one
  // each, so that every SM gets some.  (16381 tokens of 36 heads: 54 us with 8,
  // 56 with 4, 58 with 16; a plain copy of the same bytes takes 54.)
  int tt = kRopeTable / pairs < 8 ? kRopeTable / pairs : 8;
  const int even = static_cast<int>(T / (4ll * flh::sm_count()));
  if (tt > even) tt = even;
  if (tt < 1) tt = 1;
  p.tt = tt;
  const unsigned grid = static_cast<unsigned>((static_cast<int64_t>(T) + tt - 1) / tt);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return flh::launch_early(vec ? k_rope<true> : k_rope<false>, grid, kRopeThreads, 0, s, p);
}
