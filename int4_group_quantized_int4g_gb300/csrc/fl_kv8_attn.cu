// Attention over the 8-bit paged cache for few query rows: single tokens,
// drafted tokens, short chunks.
//
//   out = sum_j p_j v_j / sum_j p_j,  p_j = 2^(x_j - m),  x_j = log2(e) scale q.k_j
//
// With few rows the work is reading the cache once, so the kernel is built to
// stream it.  The rows of a kv head (query heads of its group x tokens) are
// cut into tiles of 8 or 16 rows; a unit is (sequence, kv head, row tile, 128
// tokens), the units of the whole batch lie in one line, and each CTA takes an
// equal run of them, whatever the sequences' lengths.  A tile of rows that
// several CTAs share is joined by the last of them, in CTA order.
//
// Inside a CTA each of eight warps takes 16 tokens of every unit, with a softmax
// state of its own, joined once a segment.  A warp copies its slices by TMA
// (swizzled, so that both operand reads below are free of bank conflicts) into
// a ring of its own and waits for nobody else; two CTAs fit an SM with 8 rows.
// (With one CTA, a producer warp and a ring that all warps share, reading was
// held to 3.3 TB/s by the latency of the warps' chains of work.)
// A warp's products are transposed, so that tokens
// fill the 16 rows of mma.sync and query rows its 8 columns:
//   S^T [16 tokens x 8 rows] = K q^T,   O^T [D x 8 rows] += V^T p^T.
// Codes become f16 in registers, exactly; the contraction index of either
// product may be permuted, so a lane reads 16 contiguous bytes: of its token's
// key for the first product, and of 4 tokens' values for the second, whose
// 4 x 4 bytes it transposes with byte permutes.
// Scales stay out of the operands.  q is brought to [1, 2) by a power of two a
// row (then f16 holds it with no loss that matters: 2^-25 of the row's largest
// value).  x is scaled in fp32.  A row's reference m moves only when a maximum
// has passed it by 2^8, so p reaches 2^8.  p is rounded to f16 (2^-11, against
// the output's 2^-9) after a factor 2^6 v_scale / v_ref, v_ref the largest value
// scale so far, so that it keeps its 11 bits down to 2^-20 of the largest
// weight; the accumulators are in units of v_ref.  Sums are fp32.
#include "fl_kv8_prompt.cuh"
#include "fl_tc.cuh"

using namespace flkv;

namespace {

constexpr int kTile = 128;              // tokens of a unit
constexpr int kWarps = 8;
constexpr int kRowsThreads = 32 * kWarps;
constexpr float kPScale = 64.f;         // 2^6
constexpr float kSlack = 8.f;           // a reference may lag its maximum by 2^kSlack
constexpr float kNone = -1e30f;         // the reference of a row without a token so far
// Most rows of a sequence (query heads of a kv head x tokens) that this kernel
// takes; sequences with more go to the tcgen05 kernel, in the same call.
constexpr int kFewRows = 64;

template <int D, int NT>
struct RowsCfg {
  static constexpr int kRows = 8 * NT;
  static constexpr int kCtas = NT == 1 ? 2 : 1;      // on an SM
  static constexpr int kHalf = 16 * D;               // a warp's keys (or values) of a unit
  static constexpr int kSlots = (NT == 1 ? 3 : 6) * (128 / D);
  static constexpr int kRing = kSlots * 2 * kHalf;   // of one warp
  static constexpr int kCombLd = D + 4;              // joined rows: conflict-free float2 writes
  static constexpr int kComb = kWarps * kRows * kCombLd * 4;   // over the rings, which are empty then
  static constexpr int kMlOff = kWarps * kRing;
  static constexpr int kBarOff = kMlOff + kWarps * kRows * 2 * 4;
  static constexpr int kLastOff = kBarOff + kWarps * kSlots * 8;
  static constexpr int kSmem = kLastOff + 16;
  static_assert(kComb <= kWarps * kRing && kSmem <= (232448 - 1024 * kCtas) / kCtas, "shared memory");
  static constexpr int kSlot = kRows * (D + 2);      // floats of a partial: O, then m, l of each row
};

// The units of one sequence.
struct SeqWork {
  SeqInfo q;
  int rows, rt, t0, nt;   // row tiles; first tile, tiles
  long long units;
};
template <int ROWS>
__device__ __forceinline__ SeqWork seq_work(const AttnParams& p, int b) {
  SeqWork w;
  w.q = seq_info(p.seqs, b, p.block);
  w.rows = w.q.n * p.group;
  w.rt = w.rows > p.rows_lo && w.rows <= p.rows_hi ? (w.rows + ROWS - 1) / ROWS : 0;
  w.t0 = first_seen(w.q, p.window) / kTile;
  w.nt = max(1, (w.q.kv + kTile - 1) / kTile - w.t0);   // one even without tokens: it stores the zeros
  w.units = static_cast<long long>(p.heads) * w.rt * w.nt;
  return w;
}

// A run of tiles of one (sequence, head, row tile) inside the CTA's units.
struct Segment {
  int b, h, r, t, n;          // tiles [t, t + n) of the sequence's nt
  long long first;            // unit of the row tile's first tile
};
template <int ROWS>
struct Walk {
  long long u, end, base;
  int b;
  SeqWork w;
  __device__ bool next(const AttnParams& p, Segment& s) {
    if (u >= end) return false;
    while (u >= base + w.units) {
      base += w.units;
      if (++b >= p.seqs.B) return false;
      w = seq_work<ROWS>(p, b);
    }
    const long long local = u - base, seg = local / w.nt;
    s.b = b;
    s.t = static_cast<int>(local - seg * w.nt);
    s.h = static_cast<int>(seg / w.rt);
    s.r = static_cast<int>(seg - static_cast<long long>(s.h) * w.rt);
    s.n = static_cast<int>(min(static_cast<long long>(w.nt - s.t), end - u));
    s.first = u - s.t;
    u += s.n;
    return true;
  }
};

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(v));
  return d;
}
template <int FMT, int D, int NT>
__global__ void __launch_bounds__(kRowsThreads, RowsCfg<D, NT>::kCtas)
    k_kv8_rows(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap, const AttnParams p) {
  using C = RowsCfg<D, NT>;
  constexpr int ROWS = C::kRows, NS = C::kSlots, KS = D / 16, WB = D / 16;   // WB: m tiles of O^T
  // No static shared memory: the dynamic part begins the CTA's window, on the
  // 1024-byte boundary that the swizzled tiles need (checked below).
  extern __shared__ __align__(1024) uint8_t smem[];
  float* comb = reinterpret_cast<float*>(smem);
  float* ml = reinterpret_cast<float*>(smem + C::kMlOff);          // [warp][row][m, l]
  int* s_last = reinterpret_cast<int*>(smem + C::kLastOff);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBarOff) + warp * NS;
  uint8_t* ring = smem + warp * C::kRing;
  if (smem_u32(smem) & 1023u) {
    if (tid == 0) set_status(p.status, FL_ERR_DEVICE_CHECK, 57);
    return;
  }
  if (lane == 0) {
    for (int i = 0; i < NS; ++i) mbar_init(&full[i], 1);
    fence_mbar_init();
  }
  const Start start =
      find_start<kRowsThreads>(reinterpret_cast<long long*>(smem), p.seqs.B, blockIdx.x, gridDim.x, 1,
                               [&](int b) { return seq_work<ROWS>(p, b).units; });
  const long long U = start.U;
  const int P = start.P, c = blockIdx.x;
  if (c >= P) return;
  fence_proxy_async();   // the scan's scratch lies in a ring
  __syncthreads();
  Walk<ROWS> walk;
  walk.u = unit_begin(c, U, P);
  walk.end = unit_begin(c + 1, U, P);
  walk.b = start.b;
  walk.base = start.base;
  walk.w = seq_work<ROWS>(p, walk.b);
  const long long ubeg = walk.u;

  const int g = lane >> 2, t = lane & 3;
  const int lb = 31 - __clz(p.block);   // block = 2^lb
  bool ok = true;
  int slot = 0;         // of the next slice to take
  uint32_t phase = 0;
  Segment s;
  while (walk.next(p, s)) {
    const SeqWork& w = walk.w;
    const int past = w.q.kv - w.q.n;   // position of the sequence's first row
    const int pos0 = (w.t0 + s.t) * kTile + 16 * warp;   // the warp's first token
    // ---------------- the warp's slices: lane i knows the pages of 32 of them
    const PageRun run = read_pages(w.q, p.block, p.window);
    auto page_at = [&](int i) {   // the (page, head) of slice i, -1 for none
      const int pg = (pos0 + i * kTile) >> lb;
      if (i >= s.n || pg < run.first || pg >= run.first + run.n) return -1;
      const int id = page_block(p.seqs, s.b, pg, p.num_blocks);
      if (id < 0) set_status(p.status, FL_ERR_DEVICE_CHECK, 52);
      return id < 0 ? -1 : id * p.heads + s.h;   // (blocks x heads x tokens fit 31 bits)
    };
    auto scales_of = [&](int at) { return at < 0 ? make_float2(1.f, 1.f) : make_float2(p.ks[at], p.vs[at]); };
    int ids = page_at(lane), next_ids = page_at(32 + lane);   // of the slices being copied, and the 32 after them
    int issued = 0, to = slot;                                // slices copied so far, the slot of the next
    auto copy = [&]() {
      if (issued >= s.n || !ok) return;
      const int at = __shfl_sync(0xffffffffu, ids, issued & 31);
      if (lane == 0) {
        if (at >= 0) {
          const int row = (at << lb) + ((pos0 + issued * kTile) & (p.block - 1));
          mbar_arrive_expect_tx(&full[to], 2 * C::kHalf);
          tma_load_2d(ring + to * 2 * C::kHalf, &kmap, 0, row, &full[to]);
          tma_load_2d(ring + to * 2 * C::kHalf + C::kHalf, &vmap, 0, row, &full[to]);
        } else {
          mbar_arrive(&full[to]);
        }
      }
      ++issued;
      if (++to == NS) to = 0;
    };
#pragma unroll 1
    for (int i = 0; i < NS - 1; ++i) copy();
    float2 next_scales = scales_of(ids);   // of the 32 slices being copied

    // query rows as the B operand: lane (g, t) has row g's elements [t D/4, (t+1) D/4)
    uint32_t qf[NT][KS][2];
    float fac[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = s.r * ROWS + 8 * nt + g;
      uint4 raw[D / 32];
#pragma unroll
      for (int i = 0; i < D / 32; ++i) raw[i] = make_uint4(0, 0, 0, 0);
      if (r < w.rows) {
        const int tok = r / p.group, hd = s.h * p.group + (r - tok * p.group);
        const uint4* src = reinterpret_cast<const uint4*>(p.q + (w.q.start + tok) * p.qs + static_cast<int64_t>(hd) * D + t * (D / 4));
#pragma unroll
        for (int i = 0; i < D / 32; ++i) raw[i] = src[i];
      }
      uint32_t top = 0;   // the largest magnitude's bits
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const uint32_t a[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) top = max(top, max(a[k] & 0x7fffu, (a[k] >> 16) & 0x7fffu));
      }
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int e = row_exponent(top);
      const float down = pow2i(-e);
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const uint32_t a[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
        for (int k = 0; k < 4; ++k)
          qf[nt][2 * i + (k >> 1)][k & 1] = pack_f16(__uint_as_float(a[k] << 16) * down, __uint_as_float(a[k] & 0xffff0000u) * down);
      }
      const float f = p.scale2 * pow2i(e);
#pragma unroll
      for (int h = 0; h < 2; ++h) fac[nt][h] = __shfl_sync(0xffffffffu, f, 4 * (2 * t + h));
    }
    // tokens that any row of the tile sees are [low_lo, lim_hi), that every row sees [low_hi, lim_lo)
    const int lim_lo = past + s.r * ROWS / p.group + 1;
    const int lim_hi = past + min(s.r * ROWS + ROWS - 1, w.rows - 1) / p.group + 1;
    const int low_lo = p.window ? lim_lo - p.window : 0, low_hi = p.window ? lim_hi - p.window : 0;

    float o[WB][NT][4];
    float m[NT][2], l[NT][2], vref = 0.f, rv = 0.f;   // rv: 1 / vref
#pragma unroll
    for (int i = 0; i < WB; ++i)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[i][nt][k] = 0.f;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int h = 0; h < 2; ++h) m[nt][h] = kNone, l[nt][h] = 0.f;

    float2 scales = next_scales;
#pragma unroll 1
    for (int i = 0; i < s.n; ++i) {
      if ((i & 31) == 0 && i > 0) {
        scales = next_scales;
      } else if ((i & 31) == 33 - NS && i + NS < s.n + 1) {
        // the next copy is the first of 32 more slices
        ids = next_ids;
        next_ids = page_at((i & ~31) + 64 + lane);
        next_scales = scales_of(ids);
      }
      copy();
      if (!__all_sync(0xffffffffu, ok && mbar_wait_many(&full[slot], phase))) {
        if (ok) {   // a wait ran out: nothing more is copied, the rest is walked through without data
          if (lane == 0) set_status(p.status, FL_ERR_TIMEOUT, 54);
          int sl = slot;
          uint32_t ph = phase;
          for (int k = i; k < issued; ++k) {   // (what is in flight may still land)
            mbar_wait_many(&full[sl], ph);
            if (++sl == NS) sl = 0, ph ^= 1u;
          }
        }
        ok = false;
      }
      const int pos = pos0 + i * kTile;
      const float2 sc = make_float2(__shfl_sync(0xffffffffu, scales.x, i & 31), __shfl_sync(0xffffffffu, scales.y, i & 31));
      if (ok && pos < lim_hi && pos + 16 > low_lo) {
        const uint8_t* kt = ring + slot * 2 * C::kHalf;
        const uint8_t* vt = kt + C::kHalf;
        // S^T = K q^T, in two chains
        float x[NT][4], x2[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 4; ++k) x[nt][k] = 0.f, x2[nt][k] = 0.f;
        {
          uint32_t ka[2][KS];
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int cc = 0; cc < D / 64; ++cc) {
              const uint4 v = *reinterpret_cast<const uint4*>(kt + chunk_at<D>(g + 8 * h, t * (D / 64) + cc));
              ka[h][4 * cc] = bias_codes<FMT>(v.x), ka[h][4 * cc + 1] = bias_codes<FMT>(v.y);
              ka[h][4 * cc + 2] = bias_codes<FMT>(v.z), ka[h][4 * cc + 3] = bias_codes<FMT>(v.w);
            }
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            const uint32_t a0 = code_pair_f16<FMT, false>(ka[0][k]), a2 = code_pair_f16<FMT, true>(ka[0][k]);
            const uint32_t a1 = code_pair_f16<FMT, false>(ka[1][k]), a3 = code_pair_f16<FMT, true>(ka[1][k]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma_f16(k & 1 ? x2[nt] : x[nt], a0, a1, a2, a3, qf[nt][k][0], qf[nt][k][1]);
          }
        }
        const bool mask = pos + 16 > lim_lo || pos < low_hi;
        bool grow = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 4; ++k) x[nt][k] = (x[nt][k] + x2[nt][k]) * (sc.x * fac[nt][k & 1]);
        if (mask) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int tok = pos + g + (k >> 1) * 8;
              const int lm = past + min(s.r * ROWS + 8 * nt + 2 * t + (k & 1), w.rows - 1) / p.group + 1;
              if (tok >= lm || (p.window && tok < lm - p.window)) x[nt][k] = -INFINITY;
            }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int h = 0; h < 2; ++h) grow |= fmaxf(x[nt][h], x[nt][h + 2]) > m[nt][h] + kSlack;
        if (__any_sync(0xffffffffu, grow) || sc.y > vref) {
          // a maximum has outgrown its reference, or the value scale is the largest so far
          const float vnew = fmaxf(vref, sc.y), vr = vref / vnew;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float mx = fmaxf(fmaxf(x[nt][h], x[nt][h + 2]), m[nt][h]);
              mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
              mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
              mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
              const float f = exp2_approx(m[nt][h] - mx);
              m[nt][h] = mx;
              l[nt][h] *= f;
#pragma unroll
              for (int q = 0; q < WB; ++q) {
                o[q][nt][h] *= f * vr;
                o[q][nt][h + 2] *= f * vr;
              }
            }
          vref = vnew, rv = 1.f / vnew;
        }
        const float pv = kPScale * sc.y * rv;
        uint32_t pb[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float e[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            e[k] = exp2_approx(x[nt][k] - m[nt][k & 1]);
            l[nt][k & 1] += e[k];
          }
          pb[nt][0] = transpose8x8(pack_f16(e[0] * pv, e[1] * pv));
          pb[nt][1] = transpose8x8(pack_f16(e[2] * pv, e[3] * pv));
        }
        // O^T += V^T p^T: lane (g, t) reads elements [g D/8, (g+1) D/8) of the
        // tokens 2t, 2t+1, 2t+8, 2t+9
        uint32_t vv[4][D / 32];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int row = 2 * t + (k & 1) + 8 * (k >> 1);
          if constexpr (D == 128) {
            const uint4 v = *reinterpret_cast<const uint4*>(vt + chunk_at<D>(row, g));
            vv[k][0] = v.x, vv[k][1] = v.y, vv[k][2] = v.z, vv[k][3] = v.w;
          } else {
            const uint2 v = *reinterpret_cast<const uint2*>(vt + chunk_at<D>(row, g >> 1) + 8 * (g & 1));
            vv[k][0] = v.x, vv[k][1] = v.y;
          }
        }
        if (pos + 16 > lim_hi || pos < low_lo) {
          // slots that no row sees may hold anything: as 0 they add 0 * 0
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int tok = pos + 2 * t + (k & 1) + 8 * (k >> 1);
            if (tok >= lim_hi || tok < low_lo)
#pragma unroll
              for (int q = 0; q < D / 32; ++q) vv[k][q] = 0;
          }
        }
#pragma unroll
        for (int q = 0; q < D / 32; ++q) {
          // 4 tokens x 4 elements: pairs of tokens for each element
          const uint32_t w0 = bias_codes<FMT>(vv[0][q]), w1 = bias_codes<FMT>(vv[1][q]);
          const uint32_t w2 = bias_codes<FMT>(vv[2][q]), w3 = bias_codes<FMT>(vv[3][q]);
          const uint32_t a01 = __byte_perm(w0, w1, 0x5140), a23 = __byte_perm(w0, w1, 0x7362);
          const uint32_t b01 = __byte_perm(w2, w3, 0x5140), b23 = __byte_perm(w2, w3, 0x7362);
          const uint32_t e0 = code_pair_f16<FMT, false>(a01), e1 = code_pair_f16<FMT, true>(a01);
          const uint32_t e2 = code_pair_f16<FMT, false>(a23), e3 = code_pair_f16<FMT, true>(a23);
          const uint32_t f0 = code_pair_f16<FMT, false>(b01), f1 = code_pair_f16<FMT, true>(b01);
          const uint32_t f2 = code_pair_f16<FMT, false>(b23), f3 = code_pair_f16<FMT, true>(b23);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma_f16(o[2 * q][nt], e0, e1, f0, f1, pb[nt][0], pb[nt][1]);
            mma_f16(o[2 * q + 1][nt], e2, e3, f2, f3, pb[nt][0], pb[nt][1]);
          }
        }
      }
      __syncwarp();   // the slot has been read
      if (++slot == NS) slot = 0, phase ^= 1u;
    }

    // ---------------- join the eight warps
    const float back = vref / kPScale;
    __syncthreads();   // every ring is empty: the rows go over them
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float sum = l[nt][h];
        sum += __shfl_xor_sync(0xffffffffu, sum, 4);
        sum += __shfl_xor_sync(0xffffffffu, sum, 8);
        sum += __shfl_xor_sync(0xffffffffu, sum, 16);
        const int row = 8 * nt + 2 * t + h;
        if (g == 0) reinterpret_cast<float2*>(ml)[warp * ROWS + row] = make_float2(m[nt][h] == kNone ? -INFINITY : m[nt][h], sum);
        float* dst = comb + (warp * ROWS + row) * C::kCombLd + 2 * g;
#pragma unroll
        for (int i = 0; i < WB; ++i)
          *reinterpret_cast<float2*>(dst + 16 * i) = make_float2(o[i][nt][h] * back, o[i][nt][h + 2] * back);
      }
    __syncthreads();
    // the sum of eight partial rows in shared memory, element pair d of row
    struct Joined {
      float mx, sum, ox, oy;
    };
    auto joined = [&](int row, int d) {
      const int at = d % (D / 8) / 2 * 16 + d / (D / 8) * 2;
      Joined r = {-INFINITY, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < kWarps; ++k) r.mx = fmaxf(r.mx, ml[2 * (k * ROWS + row)]);
#pragma unroll
      for (int k = 0; k < kWarps; ++k) {
        const float mk = ml[2 * (k * ROWS + row)];
        const float f = mk == -INFINITY ? 0.f : exp2_approx(mk - r.mx);
        const float2 v = *reinterpret_cast<const float2*>(comb + (k * ROWS + row) * C::kCombLd + at);
        r.sum = fmaf(f, ml[2 * (k * ROWS + row) + 1], r.sum);
        r.ox = fmaf(f, v.x, r.ox), r.oy = fmaf(f, v.y, r.oy);
      }
      return r;
    };
    auto finish = [&](const Joined& v, int row, int d) {   // the output of element pair d of a row
      const int r = s.r * ROWS + row;
      if (r >= w.rows) return;
      const int tok = r / p.group, hd = s.h * p.group + (r - tok * p.group);
      const int64_t tk = w.q.start + tok;
      const float inv = v.sum == 0.f ? 0.f : 1.f / v.sum;   // 0: no token (a NaN is not)
      *reinterpret_cast<__nv_bfloat162*>(p.out + tk * p.os + static_cast<int64_t>(hd) * D + d) =
          __floats2bfloat162_rn(v.ox * inv, v.oy * inv);
      if (d == 0 && p.lse) p.lse[tk * p.Hq + hd] = v.sum == 0.f ? -INFINITY : (v.mx + log2f(v.sum)) * kLn2;
    };
    const bool whole = s.n == w.nt;
    float* part = p.part + static_cast<size_t>(2 * c + (s.first < ubeg ? 0 : 1)) * C::kSlot;
    for (int i = tid; i < ROWS * D / 2; i += kRowsThreads) {
      const int row = i / (D / 2), d = 2 * (i - row * (D / 2));
      const Joined v = joined(row, d);
      if (whole) {
        finish(v, row, d);
      } else {
        __stcg(reinterpret_cast<float2*>(part + row * D + d), make_float2(v.ox, v.oy));
        if (d == 0) __stcg(reinterpret_cast<float2*>(part + ROWS * D + 2 * row), make_float2(v.mx, v.sum));
      }
    }
    if (!whole) {
      // The last of the CTAs that share the row tile adds them up, in CTA order:
      // warp k takes every eighth of them, then the warps are joined as above.
      const int cf = cta_of_unit(s.first, U, P), cl = cta_of_unit(s.first + w.nt - 1, U, P);
      __syncthreads();
      if (tid == 0) {
        fence_acq_rel_gpu();
        const int done = atomicAdd(&p.cnt[cf], 1);
        *s_last = done == cl - cf;
        if (*s_last) {
          fence_acq_rel_gpu();
          p.cnt[cf] = 0;
        }
      }
      __syncthreads();
      if (*s_last) {
        constexpr int kPer = ROWS * D / 128;   // float4 of O a lane
        constexpr int kLanes = D / 4;          // lanes of a row's float4 (a row is a whole number of passes, or two rows a pass)
        float4 acc[kPer];
        float am[kPer], al[kPer];
#pragma unroll
        for (int k = 0; k < kPer; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f), am[k] = -INFINITY, al[k] = 0.f;
#pragma unroll 1
        for (int cc = cf + warp; cc <= cl; cc += kWarps) {
          const float* sl = p.part + static_cast<size_t>(2 * cc + (s.first < unit_begin(cc, U, P) ? 0 : 1)) * C::kSlot;
          float4 v[kPer];
          float2 a[kPer];
#pragma unroll
          for (int k = 0; k < kPer; ++k) {
            v[k] = __ldcg(reinterpret_cast<const float4*>(sl) + k * 32 + lane);
            a[k] = __ldcg(reinterpret_cast<const float2*>(sl + ROWS * D) + (k * 32 + lane) / kLanes);
          }
#pragma unroll
          for (int k = 0; k < kPer; ++k) {
            const float nm = fmaxf(am[k], a[k].x);
            const float f = am[k] == nm ? 1.f : exp2_approx(am[k] - nm);
            const float h = a[k].x == -INFINITY ? 0.f : exp2_approx(a[k].x - nm);
            acc[k].x = fmaf(acc[k].x, f, h * v[k].x), acc[k].y = fmaf(acc[k].y, f, h * v[k].y);
            acc[k].z = fmaf(acc[k].z, f, h * v[k].z), acc[k].w = fmaf(acc[k].w, f, h * v[k].w);
            al[k] = fmaf(al[k], f, h * a[k].y);
            am[k] = nm;
          }
        }
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
          const int row = (k * 32 + lane) / kLanes, d = (k * 32 + lane) % kLanes * 4;
          float* dst = comb + (warp * ROWS + row) * C::kCombLd;
          // (the order of `joined`: pair d of a row lies at d % (D/8) / 2 * 16 + d / (D/8) * 2)
          *reinterpret_cast<float2*>(dst + d % (D / 8) / 2 * 16 + d / (D / 8) * 2) = make_float2(acc[k].x, acc[k].y);
          *reinterpret_cast<float2*>(dst + (d + 2) % (D / 8) / 2 * 16 + (d + 2) / (D / 8) * 2) = make_float2(acc[k].z, acc[k].w);
          if (d == 0) reinterpret_cast<float2*>(ml)[warp * ROWS + row] = make_float2(am[k], al[k]);
        }
        __syncthreads();
        for (int i = tid; i < ROWS * D / 2; i += kRowsThreads) {
          const int row = i / (D / 2), d = 2 * (i - row * (D / 2));
          finish(joined(row, d), row, d);
        }
      }
    }
    fence_proxy_async();   // what lay over the rings, before copies into them
    __syncthreads();
  }
}

// ------------------------------------------------------------------ host
// The codes as rows of head_dim bytes, `rows` tokens of a page of one head a box.
bool code_map(CUtensorMap* map, void* base, const fl_kv8_cache& c, int rows) {
  auto enc = flh::encode_fn();
  if (!enc) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(c.head_dim),
                              static_cast<cuuint64_t>(c.num_blocks) * c.kv_heads * c.block};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(c.head_dim)};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(c.head_dim), static_cast<cuuint32_t>(rows)};
  const cuuint32_t estr[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, base, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             c.head_dim == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int FMT, int D, int NT>
int launch_rows(const CUtensorMap& km, const CUtensorMap& vm, const AttnParams& p, cudaStream_t s) {
  using C = RowsCfg<D, NT>;
  static bool attr_done[64] = {false};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return FL_ERR_CUDA;
  if (dev >= 64 || !attr_done[dev]) {
    if (cudaFuncSetAttribute(k_kv8_rows<FMT, D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem) != cudaSuccess)
      return FL_ERR_CUDA;
    if (dev < 64) attr_done[dev] = true;
  }
  k_kv8_rows<FMT, D, NT><<<C::kCtas * flh::sm_count(), kRowsThreads, C::kSmem, s>>>(km, vm, p);
  return cudaGetLastError() == cudaSuccess ? FL_OK : FL_ERR_CUDA;
}

template <int FMT, int D>
int pick_rows(const CUtensorMap& km, const CUtensorMap& vm, const AttnParams& p, long long rows, cudaStream_t s) {
  return rows <= 8 ? launch_rows<FMT, D, 1>(km, vm, p, s) : launch_rows<FMT, D, 2>(km, vm, p, s);
}

}  // namespace

extern "C" int fl_kv8_attention_workspace(int T, int B, int Hq, int kv_heads, int head_dim, size_t* out) {
  if (!out || T < 1 || B < 1 || Hq < 1 || kv_heads < 1 || Hq % kv_heads) return FL_ERR_ARG;
  if (head_dim != 64 && head_dim != 128) return FL_ERR_UNSUPPORTED;
  // two partials a CTA: the rows that it shares with the CTAs before and after
  const bool prompt = static_cast<long long>(T) * (Hq / kv_heads) > kFewRows;
  const size_t few = 16 * (head_dim + 2);   // two CTAs an SM with 8 rows, or one with 16
  const size_t slot = prompt ? prompt_slot_floats(head_dim) : few;
  *out = kScratchOff + 2ull * flh::sm_count() * slot * 4;
  return FL_OK;
}

extern "C" int fl_kv8_attention(const void* q, int64_t q_stride, int Hq, const fl_kv8_cache* cache,
                                const fl_kv8_seqs* seqs, float scale, int window, void* out, int64_t out_stride,
                                float* lse, void* ws, size_t ws_bytes, fl_stream_t stream) {
  if (!q || !out || !ws || !flh::aligned16(q) || !flh::aligned16(out) || !flh::aligned16(ws) ||
      (reinterpret_cast<uintptr_t>(lse) & 3u))
    return FL_ERR_ARG;
  const int rc = flh::kv8_check(cache, seqs);
  if (rc != FL_OK) return rc;
  if (window >= seqs->max_blocks * cache->block) window = 0;   // hides no token
  if (Hq < 1 || Hq % cache->kv_heads || window < 0 || !(scale > -3.0e38f && scale < 3.0e38f)) return FL_ERR_ARG;
  const int64_t width = static_cast<int64_t>(Hq) * cache->head_dim;
  if (q_stride < width || out_stride < width || q_stride % 8 || out_stride % 8) return FL_ERR_ARG;
  size_t need = 0;
  fl_kv8_attention_workspace(seqs->T, seqs->B, Hq, cache->kv_heads, cache->head_dim, &need);
  if (ws_bytes < need) return FL_ERR_WORKSPACE;
  const long long rows = static_cast<long long>(seqs->max_q) * (Hq / cache->kv_heads);
  if (rows > 0x7fffffffll) return FL_ERR_UNSUPPORTED;
  CUtensorMap km, vm;
  AttnParams p;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.out = static_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  p.ks = cache->k_scale, p.vs = cache->v_scale;
  p.status = static_cast<int32_t*>(ws);
  p.cnt = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(ws) + kTicketOff);
  p.part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kScratchOff);
  p.qs = q_stride, p.os = out_stride;
  p.seqs = {seqs->cu_q, seqs->kv_lens, seqs->block_table, seqs->T, seqs->B, seqs->max_q, seqs->max_blocks};
  p.num_blocks = cache->num_blocks, p.block = cache->block, p.heads = cache->kv_heads;
  p.group = Hq / cache->kv_heads, p.Hq = Hq, p.window = window;
  p.scale2 = scale * 1.44269504088896340736f;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (rows > kFewRows) {
    if (!code_map(&km, cache->k, *cache, cache->block) || !code_map(&vm, cache->v, *cache, cache->block)) return FL_ERR_CUDA;
    // one sequence goes to the one kernel; a batch may hold both kinds
    p.rows_lo = seqs->B > 1 ? kFewRows : 0, p.rows_hi = 0x7fffffff;
    const int e = launch_prompt(km, vm, p, cache->format, cache->head_dim, s);
    if (e != FL_OK || seqs->B == 1) return e;
  }
  if (!code_map(&km, cache->k, *cache, 16) || !code_map(&vm, cache->v, *cache, 16)) return FL_ERR_CUDA;
  p.rows_lo = 0, p.rows_hi = kFewRows;
  if (cache->format == FL_KV8_E4M3)
    return cache->head_dim == 64 ? pick_rows<FL_KV8_E4M3, 64>(km, vm, p, rows, s)
                                 : pick_rows<FL_KV8_E4M3, 128>(km, vm, p, rows, s);
  return cache->head_dim == 64 ? pick_rows<FL_KV8_INT8, 64>(km, vm, p, rows, s)
                               : pick_rows<FL_KV8_INT8, 128>(km, vm, p, rows, s);
}
