// The linear in 8-bit integers for more than 16 tokens: tcgen05 over pairs of SMs.
//
// y^T = W x^T.  A pair of CTAs on two neighbouring SMs multiplies a tile of 256
// weight rows x BN tokens (tcgen05.mma kind::f16, cta_group::2, 256 x BN x 16,
// fp32 accumulators in tensor memory, 128 rows in each SM).  Work unit = (tile,
// 128 columns).  Each CTA loads its own 128 weight rows as 8-bit codes (16 KB by
// TMA) and half of the tokens (f16 codes, written by k_codes), so a token tile
// crosses to the pair once: 48 KB a unit and SM at BN = 256, not 80, where a
// unit's MMAs take 1024 cycles.  The codes become f16, exactly, on the way into
// tensor memory, where the MMA reads A: shared memory feeds B alone.  Many tokens
// are bound by the products (8190 x 4096 x 11008 410 us with the rounding of the
// tokens, 1.80 PFLOP/s), few by the weights' bytes (24 rows of a head of 128003 88 us,
// 6.1 TB/s), products of a few MB by the way in and out: 4 us before the first MMA
// (the tokens' kernel, its end and their way here), 2 us after the last.
//
// BN, a multiple of 32 up to 256, and how tiles meet pairs go by a plan (gemm_plan): the
// tiles are taken in waves, all pairs next to one another (8 token tiles by a run of
// weight tiles, for L2); the rest is taken whole, or cut into equal runs of units,
// whichever ends sooner.  Cut tiles come first, so that joining them hides behind
// whole ones.  A split tile is finished by the last pair to come, the parts added
// in the pairs' order: results do not depend on timing.  Up to BN = 128 the
// accumulator is doubled and a tile's end overlaps the next tile's MMAs.
//
// Roles in a CTA:
//   warp 0        tokens: per unit two TMA boxes of BN / 2 tokens x 64 columns
//   warp 1        tensor memory; in the pair's first CTA it issues the MMAs.  The whole warp
//                 runs the loop and one thread of it issues: operands then lie in uniform
//                 registers (eight MMAs in 150 cycles; by a lone thread in 650)
//   warp 2        weights: per unit a TMA box of 128 rows x 128 columns
//   warps 4..11   codes to f16 into a ring of A tiles in tensor memory, four warps a
//                 unit in turn (their arrivals, like the tokens' bytes, are counted on the
//                 barriers of the first CTA, where the MMAs are issued)
//   warps 12..19  accumulator times scales -> y, by TMA stores from a staging tile
//                 where y's rows start and end on 16 bytes.  They have more registers
//                 than the others: what spills comes back from L2, as shared memory
//                 leaves L1 next to nothing
#include "fl_int8.cuh"

using namespace fl8;

namespace {

constexpr int kThreads = 20 * 32;
constexpr int kConv0 = 4, kEpi0 = 12;
// Registers a thread: of the launch, and of the producers and the issuer, the
// converting warps and the epilogue (which spills its sums with 96).
constexpr int kRegs = 96, kRegsIo = 48, kRegsConv = 72, kRegsEpi = 144;
static_assert(4 * kRegsIo + 8 * kRegsConv + 8 * kRegsEpi <= 20 * kRegs, "the split draws on the launch's registers");
constexpr int kRing = 4;                       // A tiles (an even number: a slot has one group of converting warps)
constexpr int kWRing = 8;                      // weight stages, at most (4 or 8)
constexpr int kXRing = 8;                      // token stages, at most
constexpr int kRows = 128;                     // weight rows of a CTA
// Token stages (BN / 2 tokens x 128 columns f16 each, as two boxes), then weight
// stages: with few tokens, where the weights' bytes bound, the latter get more.
constexpr int kXBytes = 131072, kXBytesFew = 65536, kFew = 64;
constexpr int kWStage = kRows * kBlockK;
constexpr int kStaging = 32768;                // y: 4 KB a warp of the epilogue
constexpr int kStgOff = kXBytes + 4 * kWStage;
static_assert(kXBytesFew + 8 * kWStage == kStgOff && kFew * 128 * kXRing <= kXBytesFew, "stages");
constexpr int kScOff = kStgOff + kStaging;     // 256 token scales
constexpr int kSlotOff = kScOff + 1024;        // a split tile's parts
constexpr int kBarOff = kSlotOff + 512;
constexpr int kBars = 2 * kXRing + 2 * kWRing + 2 * kRing + 4 + 8;
constexpr int kJoin = kStgOff / 8;             // a warp's room for other pairs' parts, when the rings are done
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
  int32_t* cnt;      // [pair][rank]
  int32_t* status;
  // (in pairs of 8 bytes that are used together: with `whole` last, which shifts them by
  // one, 301 x 11008 x 4096 31.1 us, not 30.5)
  int M, N;
  int whole, tma_y;  // whether the rest's tiles are taken whole, one by each of the first pairs
  int BN, G, mtiles, ntiles;
  int xring, wshift, woff;   // token stages, log2 of the weight stages and where these lie
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
  __device__ Walk(const Params& p, int pair) : w(0), c(pair), tile(0), g0(0), g1(0), split(false) {
    u = p.whole ? min(pair, p.U / p.G) * p.G : p.U ? unit_begin(pair, p.U, p.P) : 0;
    u1 = p.whole ? min(u + p.G, p.U) : p.U ? unit_begin(pair + 1, p.U, p.P) : 0;
  }
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
// TMA load of a CTA of the pair into its own shared memory, counted on a barrier of
// either (an address of the cluster's shared memory).
__device__ __forceinline__ void tma_load_pair(void* dst, const CUtensorMap* map, int c0, int c1, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          smem_u32(dst)),
      "l"(map), "r"(c0), "r"(c1), "r"(bar)
      : "memory");
}
// The first CTA's barrier at the same place.
__device__ __forceinline__ uint32_t first_cta(const uint64_t* bar) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"(smem_u32(bar)));
  return a;
}
template <int N>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
// Arrives on the first CTA's barrier.  What the arrival hands over lies in tensor
// memory and is ordered by the fences of tcgen05, so the release need not reach
// the other SM's threads: at cluster scope it costs 2000 cycles.
__device__ __forceinline__ void arrive_first(const uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(first_cta(bar)) : "memory");
}
template <int N>
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
// Orders what this thread knows of global memory before its bulk copies from it.
__device__ __forceinline__ void fence_proxy_async_all() { asm volatile("fence.proxy.async;" ::: "memory"); }
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

template <bool FP32>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    k_int8_gemm(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap,
                const __grid_constant__ CUtensorMap ymap, const Params p) {
  extern __shared__ uint8_t raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  uint64_t* xfull = reinterpret_cast<uint64_t*>(smem + kBarOff);   // first CTA: both CTAs' tokens landed
  uint64_t* xempty = xfull + kXRing;                               // the pair's MMAs have read them
  uint64_t* wfull = xempty + kXRing;                                // weights landed
  uint64_t* wempty = wfull + kWRing;                               // 4 converting warps have read them
  uint64_t* afull = wempty + kWRing;                               // first CTA: both CTAs' A tiles are there
  uint64_t* aempty = afull + kRing;                                // the pair's MMAs have read the A tile
  uint64_t* dfull = aempty + kRing;                                // [2] accumulator final
  uint64_t* dempty = dfull + 2;                                    // [2] first CTA: both CTAs have read it out
  uint64_t* joined = dempty + 2;                                   // [8] other pairs' parts landed, for a warp
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(joined + 8);
  volatile int* flags = reinterpret_cast<volatile int*>(tmem_slot + 1);   // the epilogue's: a wait ran out; parts to join
  float* sc = reinterpret_cast<float*>(smem + kScOff);
  int* slots = reinterpret_cast<int*>(smem + kSlotOff);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_rank()), pair = blockIdx.x >> 1;
  const int accs = p.BN <= 128 ? 2 : 1;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kXRing; ++i) {
      mbar_init(&xfull[i], 1);
      mbar_init(&xempty[i], 1);
    }
    for (int i = 0; i < kWRing; ++i) {
      mbar_init(&wfull[i], 1);
      mbar_init(&wempty[i], 4);
    }
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&afull[i], 8);
      mbar_init(&aempty[i], 1);
    }
    for (int i = 0; i < 8; ++i) mbar_init(&joined[i], 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&dfull[i], 1);
      mbar_init(&dempty[i], 16);
    }
    flags[0] = 0;
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

  if (warp < kConv0) {
    regs_down<kRegsIo>();
    if (warp == 0) {
      // ---------------- tokens
      if (lane == 0) {
        pdl_wait();
        Walk k(p, pair);
        const int half = p.BN / 2;
        const uint32_t bytes = static_cast<uint32_t>(half) * 256;
        int i = 0, s = 0;   // units, stage
        uint32_t ph = 1;    // parity of its last release
        bool ok = true;
        while (ok && k.next(p)) {
          int nt, mt;
          place(p, k.tile, nt, mt);
          const int m0 = mt * p.BN + rank * half;
          for (int g = k.g0; g < k.g1; ++g, ++i) {
            if (i >= p.xring && !mbar_wait_many(&xempty[s], ph)) {
              set_status(p.status, FL_ERR_TIMEOUT, 90);
              ok = false;
              break;
            }
            if (rank == 0) mbar_arrive_expect_tx(&xfull[s], 2 * bytes);
            const uint32_t bar = first_cta(&xfull[s]);
            uint8_t* dst = smem + static_cast<uint32_t>(s) * bytes;
            tma_load_pair(dst, &xmap, g * kBlockK, m0, bar);
            tma_load_pair(dst + bytes / 2, &xmap, g * kBlockK + 64, m0, bar);
            if (++s == p.xring) s = 0, ph ^= 1u;
          }
        }
        // (the last arrivals from the pair's MMAs come in before the CTA can end)
        for (int j = 0; ok && j < min(i, p.xring); ++j) {
          if (i < p.xring) s = j, ph = 0;
          ok = mbar_wait(&xempty[s], ph);
          if (++s == p.xring) s = 0, ph ^= 1u;
        }
      }
    } else if (warp == 2) {
      // ---------------- weights: older than the kernel before this one
      if (lane == 0) {
        Walk k(p, pair);
        const int wring = 1 << p.wshift;
        int i = 0;
        bool ok = true;
        while (ok && k.next(p)) {
          int nt, mt;
          place(p, k.tile, nt, mt);
          const int n0 = nt * 2 * kRows + rank * kRows;
          for (int g = k.g0; g < k.g1; ++g, ++i) {
            const int s = i & (wring - 1);
            if (i >= wring && !mbar_wait_many(&wempty[s], static_cast<uint32_t>((i >> p.wshift) - 1) & 1u)) {
              set_status(p.status, FL_ERR_TIMEOUT, 91);
              ok = false;
              break;
            }
            mbar_arrive_expect_tx(&wfull[s], kWStage);
            tma_load_2d(smem + p.woff + s * kWStage, &wmap, g * kBlockK, n0, &wfull[s]);
          }
        }
        if (!ok)
          for (int j = i - wring; j < i; ++j) mbar_wait(&wfull[j & (wring - 1)], static_cast<uint32_t>(j >> p.wshift) & 1u);
      }
    } else if (warp == 1) {
      // ---------------- MMAs of the pair
      if (rank == 0) {   // (the whole warp runs the loop: what the MMAs take then lies in uniform registers)
        const uint32_t idesc = (1u << 4) | (static_cast<uint32_t>(p.BN >> 3) << 17) | (static_cast<uint32_t>(256 >> 4) << 24);
        const uint32_t stage = static_cast<uint32_t>(p.BN) * 128;   // bytes of this CTA's tokens of a unit
        const uint64_t desc0 = sw128_desc(smem_u32(smem));
        const bool one = elect_one();
        Walk k(p, pair);
        int i = 0, j = 0, xs = 0;   // units, tiles, token stage
        uint32_t xph = 0;
        bool ok = true, there = false;
        while (ok && k.next(p)) {
          const int acc = accs == 2 ? j & 1 : 0, use = accs == 2 ? j >> 1 : j;
          if (use > 0 && !mbar_wait_many(&dempty[acc], static_cast<uint32_t>(use - 1) & 1u)) {
            set_status(p.status, FL_ERR_TIMEOUT, 92);
            break;
          }
          const uint32_t d = tmem + acc * 128;
          for (int g = k.g0; g < k.g1; ++g, ++i) {
            const int s = i & (kRing - 1);
            if (!there && (!mbar_wait_many(&xfull[xs], xph) || !mbar_wait_many(&afull[s], static_cast<uint32_t>(i >> 2) & 1u))) {
              set_status(p.status, FL_ERR_TIMEOUT, 93);
              ok = false;
              break;
            }
            const int x = xs;
            if (++xs == p.xring) xs = 0, xph ^= 1u;
            tc_fence_after();
            if (one) {
              const uint64_t b = desc0 + ((static_cast<uint32_t>(x) * stage) >> 4);
              const uint32_t a = tmem + kACols + s * 64;
#pragma unroll
              for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                  mma_pair(d, a + h * 32 + q * 8, b + h * (stage >> 5) + q * 2, idesc, g != k.g0 || h != 0 || q != 0);
              commit_pair(&xempty[x]);
              commit_pair(&aempty[s]);
            }
            __syncwarp();
            there = mbar_test(&xfull[xs], xph) && mbar_test(&afull[(i + 1) & (kRing - 1)], static_cast<uint32_t>((i + 1) >> 2) & 1u);
          }
          if (ok && one) commit_pair(&dfull[acc]);
          __syncwarp();
          ++j;
        }
      }
    }
  } else if (warp < kEpi0) {
    regs_down<kRegsConv>();
    // ---------------- codes to f16: thread = weight row = tensor memory lane; every other unit
    const int q = warp & 3, mine = (warp - kConv0) >> 2, r = q * 32 + lane;
    const uint32_t ta = tmem + kACols + (static_cast<uint32_t>(q * 32) << 16);
    const uint8_t* rows = smem + p.woff + r * 128;
    Walk k(p, pair);
    int i = 0;
    bool ok = true;
    while (ok && k.next(p)) {
      for (int g = k.g0; g < k.g1; ++g, ++i) {
        if ((i & 1) != mine) continue;
        const int s = i & (kRing - 1), ws = i & ((1 << p.wshift) - 1);
        const uint32_t ph = static_cast<uint32_t>(i >> 2) & 1u;
        if (!mbar_wait_many(&wfull[ws], static_cast<uint32_t>(i >> p.wshift) & 1u)) {
          set_status(p.status, FL_ERR_TIMEOUT, 94);
          ok = false;
          break;
        }
        uint4 c[8];
#pragma unroll
        for (int t = 0; t < 8; ++t) c[t] = *reinterpret_cast<const uint4*>(rows + ws * kWStage + ((t ^ (r & 7)) << 4));
        __syncwarp();
        if (lane == 0) mbar_arrive(&wempty[ws]);
        if (i >= kRing && !mbar_wait_many(&aempty[s], ph ^ 1u)) {
          set_status(p.status, FL_ERR_TIMEOUT, 95);
          ok = false;
          break;
        }
        tc_fence_after();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t o[32];
#pragma unroll
          for (int t = 0; t < 16; ++t) codes_f16((&c[4 * h + (t >> 2)].x)[t & 3], o[2 * t], o[2 * t + 1]);
          tmem_st32(ta + s * 64 + h * 32, o);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_first(&afull[s]);
      }
    }
    if (ok)   // (both groups see the last arrivals in)
      for (int j = i > kRing ? i - kRing : 0; j < i; ++j)
        if ((j & 1) == mine) mbar_wait(&aempty[j & (kRing - 1)], static_cast<uint32_t>(j >> 2) & 1u);
  } else {
    regs_up<kRegsEpi>();
    // ---------------- y: weight rows 32q .. 32q + 31, half of the tile's tokens, some at a
    // time.  Tensor memory is read in mma's fragments (lane: rows g, g + 8, .. of 32,
    // tokens 2c and 2c + 1), which stmatrix turns into rows of y; a warp's staging
    // buffers have TMA's swizzle, so both sides of them are free of bank conflicts,
    // and no warp waits for another.
    constexpr int kStep = FP32 ? 16 : 32;            // tokens of a step; two buffers of 2 KB for them
    pdl_wait();
    const int e = warp - kEpi0, q = warp & 3, h = e >> 2, tid = threadIdx.x - kEpi0 * 32;
    const int g = lane >> 2, c2 = 2 * (lane & 3);
    const int mine = p.BN / 2, c0 = h * mine;        // this warp's tokens
    const int bytes = mine * 128;                    // of its part of a split tile: [16 tokens][4][lane] of 16 bytes
    int buf = 0;
    Walk k(p, pair);
    for (int j = 0; k.next(p); ++j) {
      const int acc = accs == 2 ? j & 1 : 0, use = accs == 2 ? j >> 1 : j;
      int nt, mt;
      place(p, k.tile, nt, mt);
      const int n0 = nt * 2 * kRows + rank * kRows, m0 = mt * p.BN;
      const int T = k.tile - p.waves * p.P;          // of a split tile, whose pairs are cf .. cl
      const int cf = k.split ? pair_of(T * p.G, p.U, p.P) : 0, cl = k.split ? pair_of((T + 1) * p.G - 1, p.U, p.P) : 0;
      int32_t* cnt = p.cnt + cf * 2 + rank;
      named_bar(1, 256);   // (the scales of the tile before have been used)
      if (tid < p.BN) sc[tid] = m0 + tid < p.M ? p.x_scale[m0 + tid] : 0.f;
      float ts[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int n = n0 + q * 32 + i * 8 + g;
        ts[i] = n < p.N ? __ldg(p.w_scale + n) : 0.f;
      }
      if (!mbar_wait(&dfull[acc], static_cast<uint32_t>(use) & 1u)) flags[0] = 1;
      if (tid == 0) flags[1] = k.split ? ld_acquire_gpu(cnt) == cl - cf : 1;   // the others of a split tile have all come
      named_bar(1, 256);
      if (flags[0]) {
        set_status(p.status, FL_ERR_TIMEOUT, 97);
        break;
      }
      const bool final = k.u >= k.u1 && k.w >= p.waves;   // the CTA's last tile
      bool own = flags[1] != 0;      // the sums are in tensor memory, and the others' parts have come
      tc_fence_after();
      const uint32_t d = tmem + acc * 128 + (static_cast<uint32_t>(q * 32) << 16) + c0;
      auto release = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_first(&dempty[acc]);
      };
      auto issue = [&](int t, uint32_t* u) {   // 16 tokens from t on
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint32_t* r = u + 8 * i;
          asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                       : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                       : "r"(d + (static_cast<uint32_t>(16 * i) << 16) + t));
        }
      };
      // 16 tokens from t on, as y: u[8 i + 4 b + 2 r + k] is row 16 i + 8 r + g, token t + 8 b + c2 + k
      auto scaled = [&](int t, const uint32_t* u, uint32_t* y) {
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const float2 s2 = *reinterpret_cast<const float2*>(sc + c0 + t + 8 * b + c2);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int at = 8 * (i >> 1) + 4 * b + 2 * (i & 1);
            const float f0 = __uint_as_float(u[at]) * __fmul_rn(s2.x, ts[i]), f1 = __uint_as_float(u[at + 1]) * __fmul_rn(s2.y, ts[i]);
            if constexpr (FP32) {
              y[8 * b + 2 * i] = __float_as_uint(f0), y[8 * b + 2 * i + 1] = __float_as_uint(f1);
            } else {
              const __nv_bfloat162 b2 = __floats2bfloat162_rn(f0, f1);
              y[4 * b + i] = *reinterpret_cast<const uint32_t*>(&b2);
            }
          }
        }
      };
      uint8_t* st = smem + kStgOff + e * (kStaging / 8);
      auto buffer = [&]() {   // the next one; the step before the last has left it
        st = smem + kStgOff + e * (kStaging / 8) + buf * (kStaging / 16);
        buf ^= 1;
        if (lane == 0) bulk_wait_read<1>();
        __syncwarp();
      };
      auto stage = [&](int x, const uint32_t* y) {   // tokens x .. x + 15 of the buffer
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          if constexpr (FP32) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int tok = x + 8 * b + c2 + (i & 1), n = 8 * (i >> 1) + g;
              *reinterpret_cast<uint32_t*>(st + tok * 128 + (((n >> 2) ^ (tok & 7)) << 4) + (n & 3) * 4) = y[8 * b + i];
            }
          } else {
            const int tok = x + 8 * b + (lane & 7);
            asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(
                             smem_u32(st + tok * 64 + (((lane >> 3) ^ ((tok >> 1) & 3)) << 4))),
                         "r"(y[4 * b]), "r"(y[4 * b + 1]), "r"(y[4 * b + 2]), "r"(y[4 * b + 3])
                         : "memory");
          }
        }
      };
      auto store = [&](int t, int count) {   // the buffer's tokens, t .. t + count - 1 of this warp
        const int m = m0 + c0 + t, n = n0 + q * 32;
        count = min(count, p.M - m);
        if (p.tma_y) {
          fence_proxy_async();
          __syncwarp();
          if (lane == 0) {
            if (n < p.N && count > 0) tma_store_2d(&ymap, st, n, m);
            if (n < p.N && count > 16) tma_store_2d(&ymap, st + 16 * (FP32 ? 128 : 64), n, m + 16);
            bulk_commit();
          }
        } else {   // rows of y that do not start and end on 16 bytes
          __syncwarp();
          if (n + lane < p.N)
#pragma unroll 4
            for (int tok = 0; tok < count; ++tok) {
              const size_t at = static_cast<size_t>(m + tok) * p.y_stride + n + lane;
              if constexpr (FP32)
                static_cast<float*>(p.y)[at] = *reinterpret_cast<const float*>(st + tok * 128 + (((lane >> 2) ^ (tok & 7)) << 4) + (lane & 3) * 4);
              else
                static_cast<uint16_t*>(p.y)[at] =
                    *reinterpret_cast<const uint16_t*>(st + tok * 64 + (((lane >> 3) ^ ((tok >> 1) & 3)) << 4) + (lane & 7) * 2);
            }
        }
      };
      auto landed = [&](uint32_t (&u)[16]) { tmem_ld_wait(u); };
      auto part = [&](int c) {
        return reinterpret_cast<float4*>(p.part) + (static_cast<size_t>(slots[c - cf]) * 8 + e) * (bytes / 16) + lane;
      };
      // a part of a split tile
      int others = 0;
      bool room = false;
      if (k.split) {
        if (tid <= cl - cf) {   // this CTA's parts of it, by pair
          const int c = cf + tid, which = unit_begin(c, p.U, p.P) / p.G == T ? 0 : 1;
          slots[tid] = (2 * c + which) * 2 + rank;
        }
        named_bar(1, 256);
        if (!own) {
          float4* dst = part(pair);
          uint32_t u[16];
#pragma unroll 1
          for (int t = 0; t < mine; t += 16) {
            issue(t, u);
            landed(u);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              __stcg(dst + (t / 4 + i) * 32, make_float4(__uint_as_float(u[4 * i]), __uint_as_float(u[4 * i + 1]),
                                                         __uint_as_float(u[4 * i + 2]), __uint_as_float(u[4 * i + 3])));
          }
          if (!final) release();
          named_bar(1, 256);
          if (tid == 0) flags[1] = atom_add_acq_rel_gpu(cnt, 1) == cl - cf;
          named_bar(1, 256);
          if (!flags[1]) continue;
          own = final;   // (no more MMAs: tensor memory still holds them)
        }
        if (tid == 0) *cnt = 0;
        // at the CTA's last tile the rings are empty and take the parts, all in flight at once
        others = cl - cf + 1 - own;
        room = final && others * bytes <= kJoin;
        if (room) {
          if (lane == 0) {
            fence_proxy_async_all();
            mbar_arrive_expect_tx(&joined[e], static_cast<uint32_t>(others * bytes));
            for (int c = cf, o = 0; c <= cl; ++c)
              if (!(own && c == pair)) bulk_g2s(smem + e * kJoin + bytes * o++, part(c) - lane, bytes, &joined[e]);
          }
          __syncwarp();
          if (!mbar_wait(&joined[e], 0)) set_status(p.status, FL_ERR_TIMEOUT, 98);
        }
      }
      // whole tiles, and those whose one other part lies in shared memory (a sum of two
      // has no order)
      const bool two = room && own && others == 1;
      if (!k.split || two) {
        auto add = [&](int t, uint32_t* u) {
          const float4* src = reinterpret_cast<const float4*>(smem + e * kJoin) + t * 8 + lane;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float4 f = src[32 * i];
            u[4 * i] = __float_as_uint(__uint_as_float(u[4 * i]) + f.x), u[4 * i + 1] = __float_as_uint(__uint_as_float(u[4 * i + 1]) + f.y);
            u[4 * i + 2] = __float_as_uint(__uint_as_float(u[4 * i + 2]) + f.z), u[4 * i + 3] = __float_as_uint(__uint_as_float(u[4 * i + 3]) + f.w);
          }
        };
        uint32_t ua[16], ub[16], y[16];
        issue(0, ua);
        if (16 < mine) issue(16, ub);
#pragma unroll 1
        for (int t = 0; t < mine; t += kStep) {
          landed(ua);
          if (two) add(t, ua);
          scaled(t, ua, y);
          if constexpr (FP32) {   // (16 tokens a step: the buffers hold no more)
            landed(ub);
#pragma unroll
            for (int i = 0; i < 16; ++i) ua[i] = ub[i];
            if (t + 16 >= mine)
              release();
            else if (t + 32 < mine)
              issue(t + 32, ub);
          } else {
            landed(ub);
            if (t + 16 < mine) {
              if (two) add(t + 16, ub);
              scaled(t + 16, ub, y + 8);
            }
            if (t + 32 >= mine) {
              release();
            } else {
              issue(t + 32, ua);
              if (t + 48 < mine) issue(t + 48, ub);
            }
          }
          buffer();
          stage(0, y);
          if constexpr (!FP32)
            if (t + 16 < mine) stage(16, y + 8);
          store(t, min(kStep, mine - t));
        }
        continue;
      }
#pragma unroll 1
      for (int t = 0; t < mine; t += 16) {
        uint32_t u[16];
        float v[16];
        if (own) issue(t, u);
        if (own) landed(u);
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = 0.f;
        // the pairs' order, the parts of two at once on their way
#pragma unroll 1
        for (int c = cf, o = 0; c <= cl; c += 2) {
          float4 f[2][4];
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            if (c + n > cl || (own && c + n == pair)) continue;
            if (room) {
              const float4* src = reinterpret_cast<const float4*>(smem + e * kJoin + bytes * o++) + t * 8 + lane;
#pragma unroll
              for (int i = 0; i < 4; ++i) f[n][i] = src[32 * i];
            } else {
              const float4* src = part(c + n) + t * 8;
#pragma unroll
              for (int i = 0; i < 4; ++i) f[n][i] = __ldcg(src + 32 * i);
            }
          }
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            if (c + n > cl) continue;
            if (own && c + n == pair) {
#pragma unroll
              for (int i = 0; i < 16; ++i) v[i] += __uint_as_float(u[i]);
            } else {
#pragma unroll
              for (int i = 0; i < 4; ++i) v[4 * i] += f[n][i].x, v[4 * i + 1] += f[n][i].y, v[4 * i + 2] += f[n][i].z, v[4 * i + 3] += f[n][i].w;
            }
          }
        }
        if (own && t + 16 >= mine) release();
        uint32_t y[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) u[i] = __float_as_uint(v[i]);
        scaled(t, u, y);
        buffer();
        stage(0, y);
        store(t, 16);
      }
    }
    if (lane == 0) bulk_wait0();
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

// The plan of least cycles, as far as these estimates go: a unit's MMAs take 4 BN
// cycles and 512 at least, a tile's end 16 BN where nothing overlaps it; joining two
// parts takes 3000 and 1200 for each 32 tokens, more of them 1500 a part (3000 in uneven
// runs).  BN
// = 256 moves the fewest bytes for a product and is preferred by 4% for every 32.
// Measured: 1000 x 4096 x 4096 29 us in 64 whole tiles on 76 pairs, 43 cut into 76
// runs; 301 x 11008 x 4096 29 us in 86 tiles of 160 cut into 76 runs, 33 in 129 of 128.
Plan gemm_plan(int M, int N, int K, int pairs) {
  Plan best = {};
  double least = 0;
  const int G = (K + kBlockK - 1) / kBlockK;
  const long long ntiles = (N + 2 * kRows - 1ll) / (2 * kRows);
  for (int BN = 256; BN >= 32; BN -= 32) {
    if (BN < 256 && BN >= M + 32) continue;   // (the next smaller one holds all tokens too)
    const long long mtiles = (M + BN - 1ll) / BN, tiles = mtiles * ntiles;
    const double unit = BN > 128 ? 4 * BN : 512, tail = BN > 128 ? 16 * BN : 500, cols = BN / 32, prefer = 1 + 0.04 * (256 - BN) / 32;
    auto offer = [&](double cycles, int P, int waves, long long rest, int whole) {
      cycles *= prefer;
      if (best.BN && cycles >= least) return;
      least = cycles;
      best = {BN, G, mtiles, ntiles, P, waves, rest * G, whole};
    };
    const long long q = tiles / pairs, rest = tiles % pairs;
    if (q > 0x7ffffff) continue;
    const int P = tiles < pairs ? static_cast<int>(tiles) : pairs;
    offer((q + (rest != 0)) * (G * unit + tail), P, static_cast<int>(tiles < pairs ? 0 : q), tiles < pairs ? tiles : rest, 1);
    if (rest && tiles * G >= pairs) {
      const double even = tiles * static_cast<double>(G) / pairs * unit + (q + 1) * tail;
      const double join = q > 1 ? tail : q == 1 ? 3000 + 1200 * cols : 3000 + 3000 * cols * pairs / tiles;
      offer(even + join, pairs, static_cast<int>(q ? q - 1 : 0), q ? rest + pairs : rest, 0);
    }
    for (int parts = 2; parts <= 8 && tiles * parts <= pairs && parts <= G; ++parts)
      offer((G + parts - 1) / parts * unit + tail + (parts == 2 ? 3000 + 1200 * cols : 2000 + 1500 * (parts - 1) * cols),
            static_cast<int>(tiles) * parts, 0, tiles, 0);
  }
  return best;
}
int gemm_pairs() { return flh::sm_count() / 2 < 128 ? flh::sm_count() / 2 : 128; }

size_t gemm_part_bytes(int M, int N, int K) {
  const Plan a = gemm_plan(M, N, K, gemm_pairs());
  return static_cast<size_t>(a.P) * 4 * kRows * a.BN * 4;
}

int gemm_launch(const Call& c, cudaStream_t s) {
  auto enc = flh::encode_fn();
  if (!enc) return FL_ERR_CUDA;
  Params p = {};
  p.x_scale = c.x_scale, p.w_scale = c.w_scale, p.y = c.y, p.y_stride = c.y_stride;
  p.part = c.part, p.cnt = c.cnt, p.status = c.status, p.M = c.M, p.N = c.N;
  const int pairs = gemm_pairs();
  const Plan a = pairs ? gemm_plan(c.M, c.N, c.K, pairs) : Plan{};
  if (!a.BN || a.mtiles * a.ntiles > 0x7fffffffll / kGroupM || a.units > 0x7fffffffll / (pairs + 1)) return FL_ERR_UNSUPPORTED;
  p.BN = a.BN, p.G = a.G, p.mtiles = static_cast<int>(a.mtiles), p.ntiles = static_cast<int>(a.ntiles);
  p.P = a.P, p.waves = a.waves, p.U = static_cast<int>(a.units), p.whole = a.whole;
  p.xring = kXBytes / (p.BN * 128) < kXRing ? kXBytes / (p.BN * 128) : kXRing;
  p.wshift = p.BN <= kFew ? 3 : 2;
  p.woff = p.BN <= kFew ? kXBytesFew : kXBytes;

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
  // (a swizzled store ends at whole 16 bytes: past a ragged N it would write into what lies beside y)
  p.tma_y = flh::aligned16(c.y) && c.y_stride * size % 16 == 0 && c.N * size % 16 == 0;
  memset(&ymap, 0, sizeof(ymap));
  if (p.tma_y) {
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(c.N), static_cast<cuuint64_t>(c.M)}, strides[1] = {static_cast<cuuint64_t>(c.y_stride) * size};
    const cuuint32_t box[2] = {32, 16};
    if (enc(&ymap, c.fp32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, c.y, dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, c.fp32 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) !=
        CUDA_SUCCESS)
      return FL_ERR_CUDA;
  }
  static bool ready[64] = {false};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 0 && dev < 64 && !ready[dev]) {
    cudaFuncAttributes a, b;   // the roles' register counts add up to the launch's
    if (cudaFuncGetAttributes(&a, k_int8_gemm<false>) != cudaSuccess || cudaFuncGetAttributes(&b, k_int8_gemm<true>) != cudaSuccess ||
        a.numRegs != kRegs || b.numRegs != kRegs ||
        cudaFuncSetAttribute(k_int8_gemm<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) != cudaSuccess ||
        cudaFuncSetAttribute(k_int8_gemm<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) != cudaSuccess) {
      cudaGetLastError();
      return FL_ERR_CUDA;
    }
    ready[dev] = true;
  }
  return flh::launch_early(c.fp32 ? k_int8_gemm<true> : k_int8_gemm<false>, dim3(2 * p.P), dim3(kThreads), kSmem, s, wmap, xmap, ymap, p);
}

}  // namespace fl8
