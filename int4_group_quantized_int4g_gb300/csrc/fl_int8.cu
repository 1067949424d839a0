// The linear layer in 8-bit integers: its entry points and the rounding of the
// tokens.
//
// k_codes: a CTA owns a row of x, reads it once (16 bytes a thread and load,
// kept in registers up to 32 columns a thread), takes its largest magnitude as
// integers (the bits of |bf16| order like the values), and writes the codes:
// as int8, or for the products as f16, which holds them exactly, in rows or in
// the order in which mma.sync lanes read them.  A code is the nearest whole
// number to the quotient itself: fp32's a * (127 / top) is within 2^-15 of it, and
// next to a border the sign of 2a - (2k + 1) scale decides, which one fma gives
// without a rounding that could hide it.  Large ones are bound by instructions, 19 an
// element: 8190 x 4096 to int8 27 us in a chain, where the bytes (2 + 1 an element)
// take 15; a scheduler issues in 0.70 of the cycles.  2048 x 4096 takes 10 us (bytes 3.8),
// small ones are bound by latency (1 x 4096 1.6 us, 301 x 4096 3.2).
#include "fl_int8.cuh"

using namespace fl8;

namespace {

enum { kInBf16 = 0, kInCodes = 1 };
enum { kOutCodes = 0, kOutRows = 1, kOutFrags = 2 };

struct CodesParams {
  const void* x;
  int64_t stride;
  void* out;
  float* scale;
  int M, K;
  int vec;        // rows of x may be read 16 (codes: 8) bytes at a time
  int tiles;      // kOutFrags: tiles of 8 tokens
};

// Columns 8v .. 8v+7 of a row, zeros from K on: bf16 pairs, or int8 codes in the
// first two words.
template <int IN>
__device__ __forceinline__ uint4 load8(const CodesParams& p, const void* row, int v) {
  const int k = 8 * v;
  uint4 r = make_uint4(0, 0, 0, 0);
  if (p.vec && k + 8 <= p.K) {
    if constexpr (IN == kInBf16) {
      r = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(row) + k);
    } else {
      const uint2 c = *reinterpret_cast<const uint2*>(static_cast<const int8_t*>(row) + k);
      r.x = c.x, r.y = c.y;
    }
    return r;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (k + i >= p.K) break;
    if constexpr (IN == kInBf16)
      (&r.x)[i / 2] |= static_cast<uint32_t>(static_cast<const uint16_t*>(row)[k + i]) << (16 * (i & 1));
    else
      (&r.x)[i / 4] |= static_cast<uint32_t>(static_cast<const uint8_t*>(row)[k + i]) << (8 * (i & 3));
  }
  return r;
}

// A row's quotients are x * up * inv (up: a power of two that keeps rows of tiny
// values clear of subnormal numbers, and twice the largest finite); twice: 2 * scale * up.
struct Rounding {
  float up, inv, twice;
};
// The nearest whole number to the quotient itself, next to a border too.
__device__ __noinline__ float exact_code(float x, float up, float inv, float twice) {
  const float a = fabsf(x) * up, t = a * inv, lo = floorf(t);
  const float d = __fmaf_rn(-(lo + 0.5f), twice, 2.f * a);
  const float k = d > 0.f || (d == 0.f && (static_cast<int>(lo) & 1)) ? lo + 1.f : lo;
  return copysignf(k, x);
}
// Eight values (bf16 pairs) to whole numbers.  Adding 1.5 * 2^23 rounds to them.
__device__ __forceinline__ void codes8(const uint4& r, const Rounding& q, float (&k)[8]) {
  constexpr float kMagic = 12582912.f;
  float off = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t w = (&r.x)[i / 2];
    const float t = __uint_as_float(i & 1 ? w & 0xffff0000u : w << 16) * q.up * q.inv;
    k[i] = __fsub_rn(__fadd_rn(t, kMagic), kMagic);
    off = fmaxf(off, fabsf(t - k[i]));
  }
  if (off > 0.4995f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t w = (&r.x)[i / 2];
      const float x = __uint_as_float(i & 1 ? w & 0xffff0000u : w << 16);
      if (fabsf(x * q.up * q.inv - k[i]) > 0.4995f) k[i] = exact_code(x, q.up, q.inv, q.twice);
    }
  }
}

template <int IN, int OUT, int NV>
__global__ void __launch_bounds__(1024) k_codes(const CodesParams p) {
  __shared__ uint32_t tops[32];
  const int m = blockIdx.x, tid = threadIdx.x, T = blockDim.x;
  pdl_wait();
  pdl_launch_dependents();   // (after the wait: a kernel that starts now finds all earlier ones complete)
  const int width = OUT == kOutFrags ? (p.K + kBlockK - 1) / kBlockK * kBlockK : p.K;
  const int nv = (width + 7) / 8;
  const void* row = IN == kInBf16 ? static_cast<const void*>(static_cast<const __nv_bfloat16*>(p.x) + m * p.stride)
                                  : static_cast<const void*>(static_cast<const int8_t*>(p.x) + m * p.stride);
  uint4 held[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) held[i] = tid + i * T < nv ? load8<IN>(p, row, tid + i * T) : make_uint4(0, 0, 0, 0);

  Rounding q = {1.f, 0.f, 0.f};   // (inv 0: every code is 0)
  bool none = false;
  if constexpr (IN == kInBf16) {
    uint32_t top2 = 0;   // two maxima of |bf16| bits
    auto take = [&](const uint4& r) {
#pragma unroll
      for (int j = 0; j < 4; ++j) top2 = __vmaxu2(top2, (&r.x)[j] & 0x7fff7fffu);
    };
#pragma unroll
    for (int i = 0; i < NV; ++i) take(held[i]);
    for (int v = tid + NV * T; v < nv; v += T) take(load8<IN>(p, row, v));
    uint32_t top = __reduce_max_sync(0xffffffffu, max(top2 & 0xffffu, top2 >> 16));
    if (T > 32) {
      if ((tid & 31) == 0) tops[tid >> 5] = top;
      __syncthreads();
      top = __reduce_max_sync(0xffffffffu, (tid & 31) < T / 32 ? tops[tid & 31] : 0u);
    }
    const float largest = __uint_as_float(top << 16);
    float scale = __fdiv_rn(largest, 127.f);
    if (top >= 0x7f80u) scale = __uint_as_float(0x7fc00000u);
    if (tid == 0) p.scale[m] = scale;
    none = top == 0 || top >= 0x7f80u;
    q.up = largest < 0x1p-60f ? 0x1p64f : largest > 0x1p100f ? 0x1p-64f : 1.f;
    q.inv = none ? 0.f : __fdiv_rn(127.f, largest * q.up);
    q.twice = 2.f * (scale * q.up);
  }

  auto put = [&](int v, const uint4& r) {
    if constexpr (OUT == kOutCodes) {
      float k[8] = {};
      if (!none) codes8(r, q, k);
      uint32_t c[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t b[4];   // (the sum's last byte is the code)
#pragma unroll
        for (int i = 0; i < 4; ++i) b[i] = __float_as_uint(k[4 * h + i] + 12582912.f);
        c[h] = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
      }
      int8_t* out = static_cast<int8_t*>(p.out) + static_cast<size_t>(m) * p.K + 8 * v;
      if ((p.K & 7) == 0 && (reinterpret_cast<uintptr_t>(p.out) & 7) == 0) {
        *reinterpret_cast<uint2*>(out) = make_uint2(c[0], c[1]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (8 * v + i < p.K) out[i] = static_cast<int8_t>(c[i / 4] >> (8 * (i & 3)));
      }
    } else {
      uint4 f = make_uint4(0, 0, 0, 0);
      if constexpr (IN == kInCodes) {
        codes_f16(r.x, f.x, f.y);
        codes_f16(r.y, f.z, f.w);
      } else if (!none) {
        float k[8];
        codes8(r, q, k);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const __half2 h = __floats2half2_rn(k[2 * i], k[2 * i + 1]);
          (&f.x)[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
      }
      uint8_t* out = static_cast<uint8_t*>(p.out);
      if constexpr (OUT == kOutRows) {
        *reinterpret_cast<uint4*>(out + (static_cast<size_t>(m) * p.K + 8 * v) * 2) = f;
      } else {
        // columns 32t + 16h + 8s of a run of 128: read s of half h, lane 4 (m % 8) + t
        const int j = v & 15, kb = v >> 4;
        const size_t at = ((static_cast<size_t>(kb) * p.tiles + (m >> 3)) * 4 + (j & 3)) * 512 + ((m & 7) * 4 + (j >> 2)) * 16;
        *reinterpret_cast<uint4*>(out + at) = f;
      }
    }
  };
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (tid + i * T < nv) put(tid + i * T, held[i]);
  for (int v = tid + NV * T; v < nv; v += T) put(v, load8<IN>(p, row, v));
}

template <int IN, int OUT>
int launch_codes(const CodesParams& p, cudaStream_t s) {
  const int width = OUT == kOutFrags ? (p.K + kBlockK - 1) / kBlockK * kBlockK : p.K;
  const int nv = (width + 7) / 8;
  // few rows: one vector a thread, for the shortest way through; many: four, for loads in flight
  if (p.M <= 2 * flh::sm_count() && nv <= 1024)
    return flh::launch_early(k_codes<IN, OUT, 1>, dim3(p.M), dim3((nv + 31) / 32 * 32), 0, s, p);
  int threads = ((nv + 3) / 4 + 31) / 32 * 32;
  if (threads > 1024) threads = 1024;
  return flh::launch_early(k_codes<IN, OUT, 4>, dim3(p.M), dim3(threads), 0, s, p);
}

bool aligned(const void* p, int n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

Layout layout(int M, int N, int K) {
  Layout l;
  auto up = [](size_t v) { return (v + 255) / 256 * 256; };
  const size_t rows = M <= kRowsMax ? (M + 7) / 8 * 8 : M;
  const size_t width = (static_cast<size_t>(K) + kBlockK - 1) / kBlockK * kBlockK;
  l.scale = kScratch;
  l.x = up(l.scale + static_cast<size_t>(M) * 4);
  l.part = up(l.x + rows * width * 2);
  l.bytes = l.part + up(M <= kRowsMax ? rows_part_bytes(M) : gemm_part_bytes(M, N, K));
  return l;
}

constexpr int kMost = 0x7fff0000;   // (tiles behind the last row still have 32-bit numbers)
bool linear_args(int M, int N, int K) { return M >= 1 && N >= 1 && K >= 16 && K % 16 == 0 && M <= kMost && N <= kMost && K <= kMost; }

}  // namespace

extern "C" int fl_int8_quantize(const void* x, int64_t x_stride, int M, int K, int8_t* codes, float* scale,
                                fl_stream_t stream) {
  if (!x || !codes || !scale || M < 1 || K < 1 || x_stride < K || K > 0x7fffff00 || !aligned(x, 2) || !aligned(scale, 4))
    return FL_ERR_ARG;
  // (a row's codes are written while others are still read)
  const uint64_t rows = M, width = K;
  if (flh::rows_meet(x, 2 * x_stride, 2 * width, rows, codes, 0, rows * width, 1) ||
      flh::rows_meet(x, 2 * x_stride, 2 * width, rows, scale, 0, 4 * rows, 1) ||
      flh::rows_meet(codes, 0, rows * width, 1, scale, 0, 4 * rows, 1))
    return FL_ERR_ARG;
  CodesParams p = {x, x_stride, codes, scale, M, K, aligned(x, 16) && x_stride % 8 == 0, 0};
  return launch_codes<kInBf16, kOutCodes>(p, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" int fl_int8_linear_workspace(int M, int N, int K, size_t* out) {
  if (!out || !linear_args(M, N, K)) return FL_ERR_ARG;
  *out = layout(M, N, K).bytes;
  return FL_OK;
}

extern "C" int fl_int8_linear(const void* x, int64_t x_stride, const float* x_scale, int M, int K, const int8_t* w,
                              const float* w_scale, int N, void* y, int64_t y_stride, int y_type, void* ws, size_t ws_bytes,
                              fl_stream_t stream) {
  if (!x || !w || !w_scale || !y || !ws || !linear_args(M, N, K) || x_stride < K || y_stride < N) return FL_ERR_ARG;
  if (y_type != FL_OUT_BF16 && y_type != FL_OUT_FP32) return FL_ERR_ARG;
  if (!flh::aligned16(w) || !flh::aligned16(ws) || !aligned(w_scale, 4) || !aligned(y, y_type == FL_OUT_FP32 ? 4 : 2) ||
      (x_scale ? !aligned(x_scale, 4) : !aligned(x, 2)))
    return FL_ERR_ARG;
  const Layout l = layout(M, N, K);
  if (ws_bytes < l.bytes) return FL_ERR_WORKSPACE;
  const uint64_t out = y_type == FL_OUT_FP32 ? 4 : 2, in = x_scale ? 1 : 2;
  auto under = [&](const void* p, uint64_t stride, uint64_t width, uint64_t rows) {
    return flh::rows_meet(p, stride, width, rows, y, y_stride * out, N * out, M);
  };
  if (under(x, x_stride * in, K * in, M) || under(w, 0, static_cast<uint64_t>(N) * K, 1) || under(w_scale, 0, 4ull * N, 1) ||
      (x_scale && under(x_scale, 0, 4ull * M, 1)))
    return FL_ERR_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  uint8_t* base = static_cast<uint8_t*>(ws);
  Call c;
  c.xh = base + l.x;
  c.x_scale = x_scale ? x_scale : reinterpret_cast<const float*>(base + l.scale);
  c.w = w, c.w_scale = w_scale;
  c.part = reinterpret_cast<float*>(base + l.part);
  c.cnt = reinterpret_cast<int32_t*>(base + kTicketOff);
  c.status = reinterpret_cast<int32_t*>(base);
  c.y_stride = y_stride, c.K = K, c.N = N, c.fp32 = y_type == FL_OUT_FP32;
  CodesParams p = {x, x_stride, base + l.x, reinterpret_cast<float*>(base + l.scale), M, K, 0, 0};
  p.vec = x_scale ? aligned(x, 8) && x_stride % 8 == 0 : aligned(x, 16) && x_stride % 8 == 0;
  c.M = M, c.y = y;
  if (M <= kRowsMax) {
    p.tiles = (M + 7) / 8;
    const int rc = x_scale ? launch_codes<kInCodes, kOutFrags>(p, s) : launch_codes<kInBf16, kOutFrags>(p, s);
    return rc != FL_OK ? rc : rows_launch(c, s);
  }
  const int rc = x_scale ? launch_codes<kInCodes, kOutRows>(p, s) : launch_codes<kInBf16, kOutRows>(p, s);
  return rc != FL_OK ? rc : gemm_launch(c, s);
}

extern "C" int fl_int8_test_plan(int M, int N, int K, int sms, long long* out) {
  if (!out || !linear_args(M, N, K) || sms < 2) return FL_ERR_ARG;
  const Plan a = gemm_plan(M, N, K, sms / 2);
  const long long v[8] = {a.BN, a.G, a.mtiles, a.ntiles, a.P, a.waves, a.units, a.whole};
  for (int i = 0; i < 8; ++i) out[i] = v[i];
  return FL_OK;
}
