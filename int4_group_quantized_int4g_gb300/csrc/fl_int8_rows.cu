// The linear in 8-bit integers for up to 16 tokens: the weights stream once
// through shared memory into mma.sync.
//
// Work unit = (tile of 256 weight rows, 128 columns): 32 KB by one TMA copy and
// the tokens' f16 codes of those columns (2 KB for 8 tokens, laid out in lane
// order by k_codes) by another, into a ring of stages that fills the SM's
// shared memory.  CTA c of P owns the units [c*U/P, (c+1)*U/P) in tile-major
// order, so every SM streams the same bytes.  Warp w takes rows 32w .. 32w+31 of
// a tile as the 16-row operand (two tiles of 16) and keeps their sums in
// registers over the columns, so no two warps share a sum, and the B fragments
// are read once for 32 rows.  The columns are permuted alike on both sides: lane
// t of a row holds 16 consecutive bytes, four steps of mma's K = 16.  Chunks
// 2t + h of the 128-byte swizzled row keep a quarter warp's loads (two rows) on
// different banks.  A tile that several CTAs share is finished warp by warp, by
// the last to take its ticket, partials added in CTA order.  Bound by HBM, N K bytes: a
// row of a head of 128003 x 4096 87 us with the rounding of the token, 6.0 TB/s;
// smaller products by latency (1 x 4096 x 4096 13 us: the token's kernel 3, the way to
// the first products 2, nine partials a tile).
#include "fl_int8.cuh"

using namespace fl8;

namespace {

constexpr int kTileRows = 256;
constexpr int kWarps = 8;                       // consumers, 32 rows each; warp 8 is the producer
constexpr int kThreads = (kWarps + 1) * 32;
constexpr int kWBytes = kTileRows * kBlockK;

template <int NT>   // tiles of 8 tokens
struct Cfg {
  static constexpr int kXBytes = NT * 2048;
  static constexpr int kStage = kWBytes + kXBytes;
  static constexpr int kStages = 6;
  static constexpr int kBarOff = kStages * kStage;
  static constexpr int kSmem = kBarOff + 2 * kStages * 8 + 1024;
  static_assert(kSmem <= 232448, "shared memory");
};

struct Params {
  const uint8_t* xf;
  const float* x_scale;
  const float* w_scale;
  void* y;
  int64_t y_stride;
  float* part;     // [2 P][warp][fragment order]
  int32_t* cnt;    // [P][warp]
  int32_t* status;
  int M, N, fp32;
  int G, U, P;
};

__device__ __forceinline__ int unit_begin(int c, int U, int P) { return static_cast<int>(static_cast<long long>(c) * U / P); }
__device__ __forceinline__ int cta_of(int u, int U, int P) {
  return static_cast<int>((static_cast<long long>(u + 1) * P - 1) / U);
}

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int NT>
__global__ void __launch_bounds__(kThreads, 1) k_int8_rows(const __grid_constant__ CUtensorMap wmap, const Params p) {
  using C = Cfg<NT>;
  constexpr int S = C::kStages;
  extern __shared__ uint8_t raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBarOff);
  uint64_t* empty = full + S;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = blockIdx.x;
  const int u0 = unit_begin(c, p.U, p.P), nu = unit_begin(c + 1, p.U, p.P) - u0;

  if (threadIdx.x == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], kWarps);
    }
    fence_mbar_init();
  }
  cta_sync();
  pdl_launch_dependents();

  if (warp == kWarps) {
    if (lane == 0) {
      auto weights = [&](int i) {
        const int u = u0 + i, T = u / p.G, g = u - T * p.G;
        mbar_arrive_expect_tx(&full[i % S], C::kStage);
        tma_load_2d(smem + (i % S) * C::kStage, &wmap, g * kBlockK, T * kTileRows, &full[i % S]);
      };
      auto tokens = [&](int i) {
        const int g = (u0 + i) % p.G;
        bulk_g2s(smem + (i % S) * C::kStage + kWBytes, p.xf + static_cast<size_t>(g) * C::kXBytes, C::kXBytes, &full[i % S]);
      };
      // the weights do not depend on the kernel before this one, which makes x
      // and has itself waited for all earlier ones
      const int lead = nu < S ? nu : S;
      for (int i = 0; i < lead; ++i) weights(i);
      pdl_wait();
      for (int i = 0; i < lead; ++i) tokens(i);
      int i = lead;
      for (; i < nu; ++i) {
        if (!mbar_wait(&empty[i % S], static_cast<uint32_t>(i / S - 1) & 1u)) {
          set_status(p.status, FL_ERR_TIMEOUT, 80);
          for (int j = i - S; j < i; ++j) mbar_wait(&full[j % S], static_cast<uint32_t>(j / S) & 1u);   // (no copy may outlive the CTA)
          break;
        }
        weights(i);
        tokens(i);
      }
    }
    return;
  }

  const int g = lane >> 2, t = lane & 3;
  float acc[2][NT][4] = {};
  pdl_wait();
  int T = u0 / p.G, k = u0 - T * p.G;
  bool whole = k == 0;
  for (int i = 0; i < nu; ++i) {
    const int s = i % S;
    if (!mbar_wait(&full[s], static_cast<uint32_t>(i / S) & 1u)) {
      set_status(p.status, FL_ERR_TIMEOUT, 81);
      return;
    }
    const int n0 = T * kTileRows + warp * 32;
    const bool idle = n0 >= p.N;
    const uint8_t* ws = smem + s * C::kStage + (warp * 32 + g) * 128;
    const uint8_t* xs = smem + s * C::kStage + kWBytes + lane * 16;
    if (!idle) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint4 w[4], x[NT][2];
#pragma unroll
        for (int r = 0; r < 4; ++r) w[r] = *reinterpret_cast<const uint4*>(ws + r * 1024 + (((2 * t + h) ^ g) << 4));
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int q = 0; q < 2; ++q) x[n][q] = *reinterpret_cast<const uint4*>(xs + (n * 4 + h * 2 + q) * 512);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t a[2][4];
#pragma unroll
          for (int r = 0; r < 4; ++r) codes_f16((&w[r].x)[j], a[r >> 1][r & 1], a[r >> 1][2 + (r & 1)]);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const uint32_t b0 = (&x[n][j >> 1].x)[2 * (j & 1)], b1 = (&x[n][j >> 1].x)[2 * (j & 1) + 1];
            mma_f16(acc[0][n], a[0], b0, b1);
            mma_f16(acc[1][n], a[1], b0, b1);
          }
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[s]);

    const bool last = k == p.G - 1;
    if (!last && i != nu - 1) {
      ++k;
      continue;
    }
    bool write = !idle;
    if (!(whole && last) && !idle) {
      const int cf = cta_of(T * p.G, p.U, p.P), cl = cta_of((T + 1) * p.G - 1, p.U, p.P);
      auto slot = [&](int cc) {
        const int which = unit_begin(cc, p.U, p.P) / p.G == T ? 0 : 1;
        return reinterpret_cast<float4*>(p.part) + ((static_cast<size_t>(2 * cc + which) * kWarps + warp) * 2 * NT) * 32 + lane;
      };
      float4* mine = slot(c);
#pragma unroll
      for (int j = 0; j < 2 * NT; ++j) {
        const float(&v)[4] = acc[j / NT][j % NT];
        __stcg(mine + j * 32, make_float4(v[0], v[1], v[2], v[3]));
      }
      __syncwarp();
      int got = 0;
      if (lane == 0) got = atom_add_acq_rel_gpu(p.cnt + cf * kWarps + warp, 1) == cl - cf;
      write = __shfl_sync(0xffffffffu, got, 0);
      if (write) {
        if (lane == 0) p.cnt[cf * kWarps + warp] = 0;
#pragma unroll
        for (int j = 0; j < 2 * NT; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[j / NT][j % NT][e] = 0.f;
#pragma unroll 4
        for (int cc = cf; cc <= cl; ++cc) {   // (CTA order)
          const float4* q = slot(cc);
#pragma unroll
          for (int j = 0; j < 2 * NT; ++j) {
            const float4 f = __ldcg(q + j * 32);
            float(&v)[4] = acc[j / NT][j % NT];
            v[0] += f.x, v[1] += f.y, v[2] += f.z, v[3] += f.w;
          }
        }
      }
    }
    if (write) {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int n = n0 + r * 8 + g;
        if (n >= p.N) continue;
        const float ts = __ldg(p.w_scale + n);
#pragma unroll
        for (int q = 0; q < 2 * NT; ++q) {
          const int m = (q >> 1) * 8 + 2 * t + (q & 1);
          if (m >= p.M) continue;
          const float v = acc[r >> 1][q >> 1][2 * (r & 1) + (q & 1)] * __fmul_rn(p.x_scale[m], ts);
          const size_t at = static_cast<size_t>(m) * p.y_stride + n;
          if (p.fp32)
            static_cast<float*>(p.y)[at] = v;
          else
            static_cast<__nv_bfloat16*>(p.y)[at] = __float2bfloat16_rn(v);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < 2 * NT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[j / NT][j % NT][e] = 0.f;
    if (last) ++T, k = 0, whole = true;
  }
}

template <int NT>
int launch(const Call& c, cudaStream_t s) {
  using C = Cfg<NT>;
  auto enc = flh::encode_fn();
  if (!enc) return FL_ERR_CUDA;
  CUtensorMap map;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(c.K), static_cast<cuuint64_t>(c.N)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(c.K)};
  const cuuint32_t box[2] = {kBlockK, kTileRows};
  const cuuint32_t estr[2] = {1, 1};
  if (enc(&map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<int8_t*>(c.w), dims, strides, box, estr,
          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return FL_ERR_CUDA;
  Params p = {static_cast<const uint8_t*>(c.xh), c.x_scale, c.w_scale, c.y, c.y_stride, c.part, c.cnt, c.status, c.M, c.N, c.fp32};
  const long long tiles = (static_cast<long long>(c.N) + kTileRows - 1) / kTileRows;
  p.G = (c.K + kBlockK - 1) / kBlockK;
  const long long U = tiles * p.G;
  const int sms = flh::sm_count();
  if (U > 0x7fffffffLL - 1) return FL_ERR_UNSUPPORTED;
  p.U = static_cast<int>(U);
  p.P = U < sms ? p.U : sms;
  // Few tiles: each split into equal parts, at most 16, so that the last of a
  // tile's CTAs does not add up more partials than the split has saved (1 x 1000 x 14336
  // 24 us with 4 parts, 18 with 8 or 16, 22 with 32; 16 x 2048 x 8192 20, 17, 19 and 21; 1 x
  // 1024 x 4096 12, 12, 14 and 19)
  if (tiles * 2 <= sms) {
    int parts = sms / static_cast<int>(tiles);
    if (parts > 16) parts = 16;
    if (parts > p.G) parts = p.G;
    p.P = static_cast<int>(tiles) * parts;
  }
  static bool ready[64] = {false};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 0 && dev < 64 && !ready[dev]) {
    if (cudaFuncSetAttribute(k_int8_rows<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem) != cudaSuccess) {
      cudaGetLastError();
      return FL_ERR_CUDA;
    }
    ready[dev] = true;
  }
  return flh::launch_early(k_int8_rows<NT>, dim3(p.P), dim3(kThreads), C::kSmem, s, map, p);
}

}  // namespace

namespace fl8 {

size_t rows_part_bytes(int M) {
  return static_cast<size_t>(2 * flh::sm_count()) * kTileRows * ((M + 7) / 8 * 8) * 4;
}

int rows_launch(const Call& c, cudaStream_t s) {
  return c.M <= 8 ? launch<1>(c, s) : launch<2>(c, s);
}

}  // namespace fl8
