// The linear in 8-bit integers for more than 32 tokens: tcgen05 over pairs of SMs.
//
// y^T = W x^T.  A pair of CTAs on two neighbouring SMs multiplies a tile of 256
// weight rows x BN tokens (tcgen05.mma kind::f16, cta_group::2, 256 x BN x 16,
// fp32 accumulators in tensor memory, 128 rows in each SM).  Work unit = (tile,
// 128 columns).  Each CTA loads its own 128 weight rows as 8-bit codes (16 KB by
// TMA) and half of the tokens (f16 codes, written by k_codes), so a token tile
// crosses to the pair once: 48 KB a unit and SM at BN = 256, not 80, where a
// unit's MMAs take 1024 cycles.  The codes become f16, exactly, on the way into
// tensor memory, where the MMA reads A: shared memory feeds B alone.
//
// BN is the tokens divided by the number of tiles that 256 asks for, rounded up to
// 32, so that 300 tokens cost two tiles of 160, not two of 256.  Up to 128 the
// accumulator is doubled and a tile's end overlaps the next tile's MMAs.
//
// Tiles are taken in waves, all pairs next to one another (8 token tiles by
// a run of weight tiles, for L2), as long as every pair gets a whole one; the
// rest, from one to two tiles a pair, is cut into equal runs of units, and comes
// first, so that joining its split tiles hides behind the whole ones.  A split
// tile is finished warp by warp by the last to take its ticket, the parts added
// in the pairs' order: results do not depend on timing.
//
// Roles in a CTA:
//   warp 0        tokens: per unit two TMA boxes of BN / 2 tokens x 64 columns
//   warp 1        tensor memory; in the pair's first CTA one thread issues the MMAs
//   warp 2        weights: per unit a TMA box of 128 rows x 128 columns
//   warps 4..11   codes to f16 into a ring of A tiles in tensor memory; they also wait for
//                 the unit's tokens, so the issuer probes one barrier a unit,
//                 the first CTA's, where both CTAs' warps arrive
//   warps 12..19  accumulator times scales -> y, by TMA stores from a staging tile
//                 where y's rows start on 16 bytes
#include "fl_int8.cuh"

using namespace fl8;

namespace {

constexpr int kThreads = 20 * 32;
constexpr int kConv0 = 4, kEpi0 = 12;
constexpr int kRing = 4;                       // stages of every ring
constexpr int kRows = 128;                     // weight rows of a CTA
constexpr int kXStage = 128 * 64 * 2 * 2;      // 128 tokens x 128 columns f16, as two boxes
constexpr int kWStage = kRows * kBlockK;
constexpr int kStaging = 32768;
constexpr int kWOff = kRing * kXStage;
constexpr int kStgOff = kWOff + kRing * kWStage;
constexpr int kScOff = kStgOff + kStaging;     // 256 token scales
constexpr int kBarOff = kScOff + 1024;
constexpr int kBars = 6 * kRing + 4;
constexpr int kSmem = kBarOff + kBars * 8 + 16 + 1024;
static_assert(kSmem <= 232448, "shared memory");
constexpr int kACols = 256;                    // tensor memory: accumulators [0, 256), A ring [256, 512)
constexpr int kGroupM = 8;                     // token tiles of a group

struct Params {
  const float* x_scale;
  const float* w_scale;
  void* y;
  int64_t y_stride;
  float* part;       // [pair][2][rank] slots of [column][row]
  int32_t* cnt;      // [pair][rank][warp]
  int32_t* status;
  int M, N, fp32, tma_y;
  int BN, G, mtiles, ntiles;
  int P, waves, U;   // pairs, whole tiles of each, units of the rest
};

__device__ __forceinline__ int unit_begin(int c, int U, int P) { return static_cast<int>(static_cast<long long>(c) * U / P); }
__device__ __forceinline__ int pair_of(int u, int U, int P) {
  return static_cast<int>((static_cast<long long>(u + 1) * P - 1) / U);
}

// A pair's runs of units: its share of the split tiles, then whole tiles.
struct Walk {
  int u, u1, w, c;
  int tile, g0, g1;
  bool split;
  __device__ Walk(const Params& p, int pair)
      : u(p.U ? unit_begin(pair, p.U, p.P) : 0), u1(p.U ? unit_begin(pair + 1, p.U, p.P) : 0), w(0), c(pair), tile(0), g0(0), g1(0), split(false) {}
  __device__ bool next(const Params& p) {
    if (u < u1) {
      const int t = u / p.G;
      tile = p.waves * p.P + t;
      g0 = u - t * p.G;
      g1 = min(p.G, g0 + u1 - u);
      u += g1 - g0;
      split = g1 - g0 != p.G;
      return true;
    }
    if (w >= p.waves) return false;
    tile = w++ * p.P + c;
    g0 = 0, g1 = p.G, split = false;
    return true;
  }
};
// Weight tile and token tile of a tile: groups of kGroupM token tiles, in them
// weight tiles ascending.
__device__ __forceinline__ void place(const Params& p, int tile, int& nt, int& mt) {
  const int per = kGroupM * p.ntiles, g = tile / per, rest = tile - g * per, m0 = g * kGroupM;
  const int rows = min(kGroupM, p.mtiles - m0);
  nt = rest / rows;
  mt = m0 + rest - nt * rows;
}

__device__ __forceinline__ void mma_pair(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrives on the barrier of both CTAs when the MMAs issued so far are done.
__device__ __forceinline__ void commit_pair(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                   smem_u32(bar)),
               "h"(static_cast<uint16_t>(3))
               : "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ bool wait_cluster(uint64_t* bar, uint32_t parity) { return mbar_wait_cluster(bar, parity); }

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    k_int8_gemm(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap,
                const __grid_constant__ CUtensorMap ymap, const Params p) {
  extern __shared__ uint8_t raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  uint64_t* xfull = reinterpret_cast<uint64_t*>(smem + kBarOff);   // tokens landed
  uint64_t* xempty = xfull + kRing;                                // the pair's MMAs have read them
  uint64_t* wfull = xempty + kRing;                                // weights landed
  uint64_t* wempty = wfull + kRing;                                // 8 converting warps have read them
  uint64_t* afull = wempty + kRing;                                // first CTA: both CTAs' A tiles and tokens are there
  uint64_t* aempty = afull + kRing;                                // the pair's MMAs have read the A tile
  uint64_t* dfull = aempty + kRing;                                // [2] accumulator final
  uint64_t* dempty = dfull + 2;                                    // [2] first CTA: both CTAs have read it out
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(dempty + 2);
  int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);
  float* sc = reinterpret_cast<float*>(smem + kScOff);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_rank()), pair = blockIdx.x >> 1;
  const int accs = p.BN <= 128 ? 2 : 1;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&xfull[i], 1);
      mbar_init(&xempty[i], 1);
      mbar_init(&wfull[i], 1);
      mbar_init(&wempty[i], 8);
      mbar_init(&afull[i], 16);
      mbar_init(&aempty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&dfull[i], 1);
      mbar_init(&dempty[i], 16);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "r"(512u) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  cta_sync();
  cluster_sync_all();   // (both CTAs' barriers and tensor memory are there)
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_launch_dependents();

  if (warp == 0) {
    // ---------------- tokens
    if (lane == 0) {
      pdl_wait();
      Walk k(p, pair);
      const int half = p.BN / 2;
      const uint32_t bytes = static_cast<uint32_t>(half) * 256;
      int i = 0;
      bool ok = true;
      while (ok && k.next(p)) {
        int nt, mt;
        place(p, k.tile, nt, mt);
        const int m0 = mt * p.BN + rank * half;
        for (int g = k.g0; g < k.g1; ++g, ++i) {
          const int s = i & (kRing - 1);
          if (i >= kRing && !mbar_wait(&xempty[s], static_cast<uint32_t>((i >> 2) - 1) & 1u)) {
            set_status(p.status, FL_ERR_TIMEOUT, 90);
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&xfull[s], bytes);
          tma_load_2d(smem + s * kXStage, &xmap, g * kBlockK, m0, &xfull[s]);
          tma_load_2d(smem + s * kXStage + bytes / 2, &xmap, g * kBlockK + 64, m0, &xfull[s]);
        }
      }
      if (!ok) {
        for (int j = i - kRing; j < i; ++j) mbar_wait(&xfull[j & (kRing - 1)], static_cast<uint32_t>(j >> 2) & 1u);
      } else {   // (the last arrivals from the pair's MMAs come in before the CTA can end)
        for (int j = i > kRing ? i - kRing : 0; j < i; ++j) mbar_wait(&xempty[j & (kRing - 1)], static_cast<uint32_t>(j >> 2) & 1u);
      }
    }
  } else if (warp == 2) {
    // ---------------- weights: older than the kernel before this one
    if (lane == 0) {
      Walk k(p, pair);
      int i = 0;
      bool ok = true;
      while (ok && k.next(p)) {
        int nt, mt;
        place(p, k.tile, nt, mt);
        const int n0 = nt * 2 * kRows + rank * kRows;
        for (int g = k.g0; g < k.g1; ++g, ++i) {
          const int s = i & (kRing - 1);
          if (i >= kRing && !mbar_wait(&wempty[s], static_cast<uint32_t>((i >> 2) - 1) & 1u)) {
            set_status(p.status, FL_ERR_TIMEOUT, 91);
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&wfull[s], kWStage);
          tma_load_2d(smem + kWOff + s * kWStage, &wmap, g * kBlockK, n0, &wfull[s]);
        }
      }
      if (!ok)
        for (int j = i - kRing; j < i; ++j) mbar_wait(&wfull[j & (kRing - 1)], static_cast<uint32_t>(j >> 2) & 1u);
    }
  } else if (warp == 1) {
    // ---------------- MMAs of the pair
    if (rank == 0 && lane == 0) {
      const uint32_t idesc = (1u << 4) | (static_cast<uint32_t>(p.BN >> 3) << 17) | (static_cast<uint32_t>(256 >> 4) << 24);
      const uint32_t box = static_cast<uint32_t>(p.BN) * 64;   // bytes of 64 columns of this CTA's tokens
      Walk k(p, pair);
      int i = 0, j = 0;   // units, tiles
      bool ok = true;
      while (ok && k.next(p)) {
        const int acc = accs == 2 ? j & 1 : 0, use = accs == 2 ? j >> 1 : j;
        if (use > 0 && !wait_cluster(&dempty[acc], static_cast<uint32_t>(use - 1) & 1u)) {
          set_status(p.status, FL_ERR_TIMEOUT, 92);
          break;
        }
        const uint32_t d = tmem + acc * 128;
        for (int g = k.g0; g < k.g1; ++g, ++i) {
          const int s = i & (kRing - 1);
          if (!wait_cluster(&afull[s], static_cast<uint32_t>(i >> 2) & 1u)) {
            set_status(p.status, FL_ERR_TIMEOUT, 93);
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t b = smem_u32(smem + s * kXStage), a = tmem + kACols + s * 64;
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int q = 0; q < 4; ++q)
              mma_pair(d, a + h * 32 + q * 8, sw128_desc(b + h * box + q * 32), idesc, g != k.g0 || h != 0 || q != 0);
          commit_pair(&xempty[s]);
          commit_pair(&aempty[s]);
        }
        if (ok) commit_pair(&dfull[acc]);
        ++j;
      }
    }
  } else if (warp >= kConv0 && warp < kEpi0) {
    // ---------------- codes to f16: thread = (weight row = tensor memory lane, half of the columns)
    const int q = warp & 3, h = (warp - kConv0) >> 2, r = q * 32 + lane;
    const uint32_t ta = tmem + kACols + (static_cast<uint32_t>(q * 32) << 16) + h * 32;
    Walk k(p, pair);
    int i = 0;
    bool ok = true;
    while (ok && k.next(p)) {
      for (int g = k.g0; g < k.g1; ++g, ++i) {
        const int s = i & (kRing - 1);
        const uint32_t ph = static_cast<uint32_t>(i >> 2) & 1u;
        if (!mbar_wait(&wfull[s], ph)) {
          set_status(p.status, FL_ERR_TIMEOUT, 94);
          ok = false;
          break;
        }
        const uint8_t* row = smem + kWOff + s * kWStage + r * 128;
        uint4 c[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) c[t] = *reinterpret_cast<const uint4*>(row + (((4 * h + t) ^ (r & 7)) << 4));
        __syncwarp();
        if (lane == 0) mbar_arrive(&wempty[s]);
        uint32_t o[32];
#pragma unroll
        for (int t = 0; t < 16; ++t) codes_f16((&c[t >> 2].x)[t & 3], o[2 * t], o[2 * t + 1]);
        if (i >= kRing && !mbar_wait(&aempty[s], ph ^ 1u)) {
          set_status(p.status, FL_ERR_TIMEOUT, 95);
          ok = false;
          break;
        }
        tc_fence_after();
        tmem_st32(ta + s * 64, o);
        tmem_wait_st();
        if (!mbar_wait(&xfull[s], ph)) {
          set_status(p.status, FL_ERR_TIMEOUT, 96);
          ok = false;
          break;
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote_rank0(&afull[s]);
      }
    }
    if (ok)
      for (int j = i > kRing ? i - kRing : 0; j < i; ++j) mbar_wait(&aempty[j & (kRing - 1)], static_cast<uint32_t>(j >> 2) & 1u);
  } else if (warp >= kEpi0) {
    // ---------------- y: rows q * 32 + lane, one half of the tokens
    pdl_wait();
    const int e = warp - kEpi0, q = warp & 3, h = e >> 2, r = q * 32 + lane, tid = threadIdx.x - kEpi0 * 32;
    const uint32_t quad = static_cast<uint32_t>(q * 32) << 16;
    Walk k(p, pair);
    for (int j = 0; k.next(p); ++j) {
      const int acc = accs == 2 ? j & 1 : 0, use = accs == 2 ? j >> 1 : j;
      int nt, mt;
      place(p, k.tile, nt, mt);
      const int n = nt * 2 * kRows + rank * kRows + r, m0 = mt * p.BN;
      named_bar(1, 256);   // (the scales of the tile before have been used)
      if (tid < p.BN) sc[tid] = m0 + tid < p.M ? p.x_scale[m0 + tid] : 0.f;
      const float ts = n < p.N ? __ldg(p.w_scale + n) : 0.f;
      if (!mbar_wait(&dfull[acc], static_cast<uint32_t>(use) & 1u)) *abort_flag = 1;
      named_bar(1, 256);
      if (*reinterpret_cast<volatile int*>(abort_flag)) {
        set_status(p.status, FL_ERR_TIMEOUT, 97);
        break;
      }
      tc_fence_after();
      const uint32_t d = tmem + acc * 128 + quad;
      auto release = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote_rank0(&dempty[acc]);
      };
      auto store16 = [&](int col, const float (&v)[16]) {   // without staging
        if (n >= p.N) return;
#pragma unroll
        for (int t = 0; t < 16; ++t) {
          if (m0 + col + t >= p.M) break;
          const float f = v[t] * __fmul_rn(sc[col + t], ts);
          const size_t at = static_cast<size_t>(m0 + col + t) * p.y_stride + n;
          if (p.fp32)
            static_cast<float*>(p.y)[at] = f;
          else
            static_cast<__nv_bfloat16*>(p.y)[at] = __float2bfloat16_rn(f);
        }
      };
      auto load16 = [&](int col, float (&v)[16]) {
        uint32_t u[16];
        tmem_ld16_issue(d + col, u);
        tmem_ld_wait(u);
#pragma unroll
        for (int t = 0; t < 16; ++t) v[t] = __uint_as_float(u[t]);
      };
      const int mine = p.BN / 2, c0 = h * mine;   // this warp's columns, without staging
      if (!k.split && p.tma_y) {
        const int round = p.fp32 ? 64 : 128;      // tokens of a staging tile
        for (int t0 = 0; t0 < p.BN; t0 += round) {
          const int n_t = min(round, p.BN - t0), lt = h * (n_t / 2);
#pragma unroll 1
          for (int col = 0; col < n_t / 2; col += 16) {
            float v[16];
            load16(t0 + lt + col, v);
            uint8_t* st = smem + kStgOff;
#pragma unroll
            for (int t = 0; t < 16; ++t) {
              const float f = v[t] * __fmul_rn(sc[t0 + lt + col + t], ts);
              const int at = (lt + col + t) * kRows + r;
              if (p.fp32)
                reinterpret_cast<float*>(st)[at] = f;
              else
                reinterpret_cast<__nv_bfloat16*>(st)[at] = __float2bfloat16_rn(f);
            }
          }
          if (t0 + round >= p.BN) release();
          fence_proxy_async();
          named_bar(1, 256);
          if (e == 0 && lane == 0) {
            for (int t = 0; t < n_t && m0 + t0 + t < p.M && n < p.N; t += 32)   // (n: the tile's first row here)
              tma_store_2d(&ymap, smem + kStgOff + t * kRows * (p.fp32 ? 4 : 2), nt * 2 * kRows + rank * kRows, m0 + t0 + t);
            bulk_commit();
            bulk_wait_read0();
          }
          named_bar(1, 256);
        }
        continue;
      }
      if (!k.split) {
#pragma unroll 1
        for (int col = c0; col < c0 + mine; col += 16) {
          float v[16];
          load16(col, v);
          if (col + 16 >= c0 + mine) release();
          store16(col, v);
        }
        continue;
      }
      // a part of a split tile: pairs cf .. cl, added in their order by the last
      const int T = k.tile - p.waves * p.P;
      const int cf = pair_of(T * p.G, p.U, p.P), cl = pair_of((T + 1) * p.G - 1, p.U, p.P);
      auto slot = [&](int c) {
        const int which = unit_begin(c, p.U, p.P) / p.G == T ? 0 : 1;
        return p.part + (static_cast<size_t>(2 * c + which) * 2 + rank) * kRows * p.BN + r;
      };
      {
        float* dst = slot(pair);
#pragma unroll 1
        for (int col = c0; col < c0 + mine; col += 16) {
          float v[16];
          load16(col, v);
          if (col + 16 >= c0 + mine) release();
#pragma unroll
          for (int t = 0; t < 16; ++t) __stcg(dst + static_cast<size_t>(col + t) * kRows, v[t]);
        }
      }
      __syncwarp();
      int last = 0;
      int32_t* cnt = p.cnt + (cf * 2 + rank) * 8 + e;
      if (lane == 0) last = atom_add_acq_rel_gpu(cnt, 1) == cl - cf;
      last = __shfl_sync(0xffffffffu, last, 0);
      if (!last) continue;
      if (lane == 0) *cnt = 0;
      __syncwarp();
#pragma unroll 1
      for (int col = c0; col < c0 + mine; col += 16) {
        float v[16];
#pragma unroll
        for (int t = 0; t < 16; ++t) v[t] = 0.f;
        for (int c = cf; c <= cl; ++c) {
          const float* src = slot(c) + static_cast<size_t>(col) * kRows;
#pragma unroll
          for (int t = 0; t < 16; ++t) v[t] += __ldcg(src + t * kRows);
        }
        store16(col, v);
      }
    }
    if (e == 0 && lane == 0) bulk_wait0();
  }
  tc_fence_before();
  __syncwarp();
  cluster_sync_all();   // (the other CTA's MMAs and arrivals are over)
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
  }
}

}  // namespace

namespace fl8 {

int gemm_bn(int M) {
  const int tiles = (M + 255) / 256;
  return ((M + tiles - 1) / tiles + 31) / 32 * 32;
}

size_t gemm_part_bytes(int M) {
  return static_cast<size_t>(flh::sm_count() / 2) * 4 * kRows * gemm_bn(M) * 4;
}

int gemm_launch(const Call& c, cudaStream_t s) {
  auto enc = flh::encode_fn();
  if (!enc) return FL_ERR_CUDA;
  Params p = {};
  p.x_scale = c.x_scale, p.w_scale = c.w_scale, p.y = c.y, p.y_stride = c.y_stride;
  p.part = c.part, p.cnt = c.cnt, p.status = c.status, p.M = c.M, p.N = c.N, p.fp32 = c.fp32;
  p.BN = gemm_bn(c.M);
  p.G = (c.K + kBlockK - 1) / kBlockK;
  p.mtiles = (c.M + p.BN - 1) / p.BN;
  p.ntiles = static_cast<int>((c.N + 2 * kRows - 1ll) / (2 * kRows));
  const long long tiles = static_cast<long long>(p.mtiles) * p.ntiles;
  if (tiles > 0x7fffffffll / kGroupM || p.ntiles > 0x7fffffff / kGroupM) return FL_ERR_UNSUPPORTED;
  const int pairs = flh::sm_count() / 2;
  p.P = pairs;
  if (tiles * 2 <= pairs) {   // few tiles: each in equal parts
    int parts = pairs / static_cast<int>(tiles);
    if (parts > 8) parts = 8;
    if (parts > p.G) parts = p.G;
    p.P = static_cast<int>(tiles) * parts;
  } else if (tiles < pairs && tiles * p.G < pairs) {
    p.P = static_cast<int>(tiles);
  }
  p.waves = static_cast<int>(tiles / p.P);
  if (tiles % p.P && p.waves) --p.waves;
  const long long U = (tiles - static_cast<long long>(p.waves) * p.P) * p.G;
  if (U > 0x7fffffffll / (pairs + 1)) return FL_ERR_UNSUPPORTED;
  p.U = static_cast<int>(U);

  const cuuint32_t estr[2] = {1, 1};
  CUtensorMap wmap, xmap, ymap;
  {
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(c.K), static_cast<cuuint64_t>(c.N)}, strides[1] = {static_cast<cuuint64_t>(c.K)};
    const cuuint32_t box[2] = {kBlockK, kRows};
    if (enc(&wmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<int8_t*>(c.w), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return FL_ERR_CUDA;
  }
  {
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(c.K), static_cast<cuuint64_t>(c.M)}, strides[1] = {static_cast<cuuint64_t>(c.K) * 2};
    const cuuint32_t box[2] = {64, static_cast<cuuint32_t>(p.BN / 2)};
    if (enc(&xmap, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, const_cast<void*>(c.xh), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return FL_ERR_CUDA;
  }
  const size_t size = c.fp32 ? 4 : 2;
  p.tma_y = flh::aligned16(c.y) && c.y_stride * size % 16 == 0;
  memset(&ymap, 0, sizeof(ymap));
  if (p.tma_y) {
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(c.N), static_cast<cuuint64_t>(c.M)}, strides[1] = {static_cast<cuuint64_t>(c.y_stride) * size};
    const cuuint32_t box[2] = {kRows, 32};
    if (enc(&ymap, c.fp32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, c.y, dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) !=
        CUDA_SUCCESS)
      return FL_ERR_CUDA;
  }
  static bool ready[64] = {false};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 0 && dev < 64 && !ready[dev]) {
    if (cudaFuncSetAttribute(k_int8_gemm, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) != cudaSuccess) {
      cudaGetLastError();
      return FL_ERR_CUDA;
    }
    ready[dev] = true;
  }
  return flh::launch_early(k_int8_gemm, dim3(2 * p.P), dim3(kThreads), kSmem, s, wmap, xmap, ymap, p);
}

}  // namespace fl8
