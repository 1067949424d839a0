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
// a ring of its own and waits for nobody else; two CTAs fit an SM.
// The copies run on into the CTA's next segment while this one is joined: the
// segments lie in shared memory one ahead.
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
// the output's 2^-8) after a factor 2^6 v_scale / v_ref, v_ref the largest value
// scale so far, so that it keeps its 11 bits down to 2^-20 of the largest
// weight; the accumulators are in units of v_ref.  Sums are fp32.
//
// Measured: 19 sequences of 65536 tokens, 8 kv heads of 128 (2.55 GB), 435 us,
// 5.9 TB/s; 48 sequences of 130 to 8100 tokens (390 MB) 77 us in a chain of
// calls, 5.1 TB/s.  What a call pays beside its bytes is the plan before the
// first copy (5 us: lengths, the CTA's units, its pages) and the joins after the
// last (4 us).
#include "fl_kv8_prompt.cuh"
#include "fl_tc.cuh"

using namespace flkv;

namespace {

constexpr int kTile = 128;              // tokens of a unit
constexpr int kWarps = 8;
constexpr int kRowsThreads = 32 * kWarps;
constexpr float kPScale = 64.f;         // 2^6
constexpr float kSlack = 8.f;           // a reference may lag its maximum by 2^kSlack
constexpr float kNone = -3.4028234663852886e38f;   // the reference of a row without a token so far: below every finite score
// Most rows of a sequence (query heads of a kv head x tokens) that this kernel
// takes; sequences with more go to the tcgen05 kernel, in the same call.  (16
// sequences of 4096 tokens, 8 heads of 128: with 24 rows 78 us here and 89 us
// there, with 32 rows 95 and 89, with 48 rows 126 and 89; 16 of 1000 tokens, 2
// heads, 32 rows: 23 and 37; one of 32768 tokens, 8 heads, 32 rows: 50 and 60.)
constexpr int kFewRows = 32;

// Up to so many CTAs of a row tile are added up by a thread for each four
// elements, more of them warp by warp and then across the warps (one sequence of
// 517 tokens, five CTAs: 9.1 us against 10.0; 12 row tiles of 25 CTAs: 65.4 us
// against 63.4).
constexpr int kDirect = 8;

template <int D, int NT>
struct RowsCfg {
  static constexpr int kRows = 8 * NT;
  static constexpr int kCtas = 2;                    // on an SM
  static constexpr int kHalf = 16 * D;               // a warp's keys (or values) of a unit
  static constexpr int kSlots = D == 128 ? 3 : NT == 1 ? 6 : 5;
  static constexpr int kRing = kSlots * 2 * kHalf;   // of one warp
  static constexpr int kVals = kRows * D / 32;       // accumulators of a lane
  static constexpr int kJoinOff = kWarps * kRing;    // four warps' accumulators, [warp][value][lane]
  static constexpr int kMlOff = kJoinOff + kWarps / 2 * kVals * 32 * 4;   // and references and sums, [warp][row]
  static constexpr int kBarOff = kMlOff + kWarps / 2 * kRows * 2 * 4;
  static constexpr int kDescOff = kBarOff + kWarps * kSlots * 8;
  static constexpr int kWalkOff = kDescOff + 3 * 64;
  static constexpr int kLastOff = kWalkOff + 96;
  static constexpr int kSmem = kLastOff + 16;
  static_assert(kSmem <= (232448 + 1024) / kCtas - 1024, "shared memory");
  static constexpr int kSlot = kRows * (D + 2);      // floats of a partial: O [4 values][lane], then m, l of each row
};

// The units of one sequence.  A row tile counts kEnd more than it has tiles:
// its start and its join take a CTA about that long, and runs of short
// sequences would take longer than others otherwise (48 sequences of 130 to
// 8100 tokens, sorted by length: 128 us without, 97 us with).
constexpr int kEnd = 2;
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
  w.units = static_cast<long long>(p.heads) * w.rt * (w.nt + kEnd);
  return w;
}

// A run of tiles of one (sequence, head, row tile) inside the CTA's units.
struct __align__(16) Segment {
  int n;                  // tiles, 0: no more segments
  int b, h, r;            // sequence, kv head, row tile
  int pos;                // first token of the first tile
  int start, past, rows;  // the sequence's first query row, its position, its rows
  int page0, pages;       // pages that a row sees
  int slot;               // the partial to write, or -1: the row tile is whole, write its output
  int cf, cl;             // CTAs that share the row tile
  int pad[3];
};
static_assert(sizeof(Segment) == 64, "segments");
template <int ROWS>
struct Walk {
  long long u, end, base, beg, U;
  int b, P;
  SeqWork w;
  __device__ void next(const AttnParams& p, Segment& s) {
    s.n = 0;
    long long seg;
    int t;
    for (;;) {
      if (u >= end) return;
      while (u >= base + w.units) {
        base += w.units;
        if (++b >= p.seqs.B) return;
        w = seq_work<ROWS>(p, b);
      }
      const long long local = u - base;
      seg = local / (w.nt + kEnd);
      t = static_cast<int>(local - seg * (w.nt + kEnd));
      if (t < w.nt) break;
      u += w.nt + kEnd - t;   // what is left of a row tile's last units
    }
    s.n = static_cast<int>(min(static_cast<long long>(w.nt - t), end - u));
    s.b = b;
    s.h = static_cast<int>(seg / w.rt);
    s.r = static_cast<int>(seg - static_cast<long long>(s.h) * w.rt);
    s.pos = (w.t0 + t) * kTile;
    s.start = w.q.start, s.past = w.q.kv - w.q.n, s.rows = w.rows;
    const PageRun run = read_pages(w.q, p.block, p.window);
    s.page0 = run.first, s.pages = run.n;
    const long long first = u - t;
    s.slot = s.n == w.nt ? -1 : 2 * static_cast<int>(blockIdx.x) + (first < beg ? 0 : 1);
    s.cf = cta_of_unit(first, U, P), s.cl = cta_of_unit(first + w.nt - 1, U, P);
    u += s.n;
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
  float* jv = reinterpret_cast<float*>(smem + C::kJoinOff);
  float2* jm = reinterpret_cast<float2*>(smem + C::kMlOff);
  Segment* segs = reinterpret_cast<Segment*>(smem + C::kDescOff);
  Walk<ROWS>* plan = reinterpret_cast<Walk<ROWS>*>(smem + C::kWalkOff);
  static_assert(sizeof(Walk<ROWS>) <= 96, "plan");
  int* s_last = reinterpret_cast<int*>(smem + C::kLastOff);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBarOff) + warp * NS;
  uint8_t* ring = smem + warp * C::kRing;
  pdl_launch_dependents();
  if (tid == 0) prefetch_map(&kmap), prefetch_map(&vmap);
  if (lane == 0) {
    for (int i = 0; i < NS; ++i) mbar_init(&full[i], 1);
    fence_mbar_init();
  }
  pdl_wait();
  if (smem_u32(smem) & 1023u) {
    if (tid == 0) set_status(p.status, FL_ERR_DEVICE_CHECK, 57);
    return;
  }
  {
    const Start start =
        find_start<kRowsThreads>(reinterpret_cast<long long*>(smem + C::kJoinOff), p.seqs.B, blockIdx.x, gridDim.x, 1,
                                 [&](int b) {
                                   const SeqWork w = seq_work<ROWS>(p, b);
                                   if (w.q.bad && blockIdx.x == 0) set_status(p.status, FL_ERR_DEVICE_CHECK, 58);
                                   return w.units;
                                 });
    if (static_cast<int>(blockIdx.x) >= start.P) return;
    if (tid == 0) {
      Walk<ROWS> walk;
      walk.U = start.U, walk.P = start.P;
      walk.u = walk.beg = unit_begin(blockIdx.x, start.U, start.P);
      walk.end = unit_begin(blockIdx.x + 1, start.U, start.P);
      walk.b = start.b;
      walk.base = start.base;
      walk.w = seq_work<ROWS>(p, walk.b);
      walk.next(p, segs[0]);
      walk.next(p, segs[1]);
      *plan = walk;
    }
    __syncthreads();
  }

  const int g = lane >> 2, t = lane & 3;
  const int lb = 31 - __clz(p.block);   // block = 2^lb
  bool ok = true;
  int slot = 0;         // of the next slice to take
  uint32_t phase = 0;
  // ---------------- the warp's slices: lane i knows the pages of 32 of them
  auto page_at = [&](const Segment& s, int i) {   // the (page, head) of slice i, -1 for none
    const int pg = (s.pos + 16 * warp + i * kTile) >> lb;
    if (i >= s.n || pg < s.page0 || pg >= s.page0 + s.pages) return -1;
    const int id = page_block(p.seqs, s.b, pg, p.num_blocks);
    if (id < 0) set_status(p.status, FL_ERR_DEVICE_CHECK, 52);
    return id < 0 ? -1 : id * p.heads + s.h;   // (blocks x heads x tokens fit 31 bits)
  };
  auto scales_of = [&](int at) { return at < 0 ? make_float2(1.f, 1.f) : make_float2(p.ks[at], p.vs[at]); };
  // Copies: of segment `on`, its `todo` slices from `from`, `issued` of them so
  // far; the pages of 32 of them and of the 32 after; the slot of the next.
  int on = 0, todo = segs[0].n, from = segs[0].pos + 16 * warp, issued = 0, to = 0;
  int ids = page_at(segs[0], lane), next_ids = page_at(segs[0], 32 + lane);
  int seg_ids = page_at(segs[1], lane);                       // the first pages of the segment after
  float2 next_scales = scales_of(ids), seg_scales;            // of the 32 slices being copied; of the next segment's first
  auto copy = [&]() {
    if (!ok || issued >= todo) return;
    const int at = __shfl_sync(0xffffffffu, ids, issued & 31);
    if (lane == 0) {
      if (at >= 0) {
        const int row = (at << lb) + ((from + issued * kTile) & (p.block - 1));
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

#pragma unroll 1
  for (int seg = 0; segs[seg % 3].n > 0; ++seg) {
    const Segment& s = segs[seg % 3];
    const int n = s.n, rows = s.rows, past = s.past;
    const int pos0 = s.pos + 16 * warp;   // the warp's first token
    if (tid == 0) {   // the segment after the next
      Walk<ROWS> walk = *plan;
      walk.next(p, segs[(seg + 2) % 3]);
      *plan = walk;
    }
    // query rows as the B operand: lane (g, t) has row g's elements [t D/4, (t+1) D/4)
    uint32_t qf[NT][KS][2];
    float fac[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = s.r * ROWS + 8 * nt + g;
      uint4 raw[D / 32];
#pragma unroll
      for (int i = 0; i < D / 32; ++i) raw[i] = make_uint4(0, 0, 0, 0);
      if (r < rows) {
        const int tok = r / p.group, hd = s.h * p.group + (r - tok * p.group);
        const uint4* src = reinterpret_cast<const uint4*>(p.q + static_cast<int64_t>(s.start + tok) * p.qs + static_cast<int64_t>(hd) * D + t * (D / 4));
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
    const int lim_hi = past + min(s.r * ROWS + ROWS - 1, rows - 1) / p.group + 1;
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

    float2 scales = seg == 0 ? next_scales : seg_scales;
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      if ((i & 31) == 0 && i > 0) scales = next_scales;
      if (on == seg && issued == todo) {
        // on to the next segment (its last slice has been issued at least an iteration ago)
        ++on;
        const Segment& x = segs[on % 3];
        todo = x.n, from = x.pos + 16 * warp, issued = 0;
        ids = seg_ids, next_ids = page_at(x, 32 + lane);
        seg_scales = scales_of(ids);
      } else if (issued > 0 && (issued & 31) == 0) {
        // the next copy is the first of 32 more slices
        ids = next_ids;
        next_ids = page_at(segs[on % 3], issued + 32 + lane);
        next_scales = scales_of(ids);
      }
      copy();
      if (!__all_sync(0xffffffffu, ok && mbar_wait_many(&full[slot], phase))) {
        if (ok) {   // a wait ran out: nothing more is copied, the rest is walked through without data
          if (lane == 0) set_status(p.status, FL_ERR_TIMEOUT, 54);
          int sl = slot;
          uint32_t ph = phase;
          do {   // (what is in flight may still land)
            mbar_wait_many(&full[sl], ph);
            if (++sl == NS) sl = 0, ph ^= 1u;
          } while (sl != to);
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
              const int lm = past + min(s.r * ROWS + 8 * nt + 2 * t + (k & 1), rows - 1) / p.group + 1;
              if (tok >= lm || (p.window && tok < lm - p.window)) x[nt][k] = -INFINITY;
            }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int h = 0; h < 2; ++h) grow |= fmaxf(x[nt][h], x[nt][h + 2]) - m[nt][h] > kSlack;   // (the difference is exact where it counts)
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

    // ---------------- join the eight warps: in three rounds, half of them hand
    // their accumulators to the others
    const float back = vref / kPScale;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        l[nt][h] += __shfl_xor_sync(0xffffffffu, l[nt][h], 4);
        l[nt][h] += __shfl_xor_sync(0xffffffffu, l[nt][h], 8);
        l[nt][h] += __shfl_xor_sync(0xffffffffu, l[nt][h], 16);
#pragma unroll
        for (int q = 0; q < WB; ++q) o[q][nt][h] *= back, o[q][nt][h + 2] *= back;
      }
    auto merge = [&](float (&f)[NT][2], float (&fo)[NT][2], const float2 (&other)[NT][2]) {   // factors of ours and theirs
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float mx = fmaxf(m[nt][h], other[nt][h].x);
          f[nt][h] = exp2_approx(m[nt][h] - mx), fo[nt][h] = exp2_approx(other[nt][h].x - mx);
          m[nt][h] = mx;
          l[nt][h] = fmaf(l[nt][h], f[nt][h], other[nt][h].y * fo[nt][h]);
        }
    };
    auto join = [&]() {   // leaves the sum in warp 0
#pragma unroll 1
      for (int half = kWarps / 2; half > 0; half >>= 1) {
        __syncthreads();   // the places have been read
        if (warp >= half && warp < 2 * half) {
          float* dst = jv + (warp - half) * C::kVals * 32 + lane;
#pragma unroll
          for (int q = 0; q < WB; ++q)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int k = 0; k < 4; ++k) dst[((q * NT + nt) * 4 + k) * 32] = o[q][nt][k];
          if (g == 0)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int h = 0; h < 2; ++h) jm[(warp - half) * ROWS + 8 * nt + 2 * t + h] = make_float2(m[nt][h], l[nt][h]);
        }
        __syncthreads();
        if (warp < half) {
          float2 other[NT][2];
          float f[NT][2], fo[NT][2];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int h = 0; h < 2; ++h) other[nt][h] = jm[warp * ROWS + 8 * nt + 2 * t + h];
          merge(f, fo, other);
          const float* src = jv + warp * C::kVals * 32 + lane;
#pragma unroll
          for (int q = 0; q < WB; ++q)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int k = 0; k < 4; ++k)
                o[q][nt][k] = fmaf(o[q][nt][k], f[nt][k & 1], src[((q * NT + nt) * 4 + k) * 32] * fo[nt][k & 1]);
        }
      }
    };
    auto output = [&]() {   // warp 0: the rows' output
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = s.r * ROWS + 8 * nt + 2 * t + h;
          if (r >= rows) continue;
          const int tok = r / p.group, hd = s.h * p.group + (r - tok * p.group);
          const int64_t tk = s.start + tok;
          const float sum = l[nt][h], inv = sum == 0.f ? 0.f : 1.f / sum;   // 0: no token (a NaN is not)
          uint32_t v[WB];
#pragma unroll
          for (int q = 0; q < WB; ++q) {   // elements g D/8 + 2 q and the next
            const __nv_bfloat162 z = __floats2bfloat162_rn(o[q][nt][h] * inv, o[q][nt][h + 2] * inv);
            v[q] = *reinterpret_cast<const uint32_t*>(&z);
          }
          uint4* dst = reinterpret_cast<uint4*>(p.out + tk * p.os + static_cast<int64_t>(hd) * D + g * (D / 8));
#pragma unroll
          for (int q = 0; q < WB / 4; ++q) dst[q] = make_uint4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
          if (g == 0 && p.lse) p.lse[tk * p.Hq + hd] = sum == 0.f ? -INFINITY : (m[nt][h] + log2f(sum)) * kLn2;
        }
    };
    join();
    if (s.slot < 0) {
      if (warp == 0) output();
    } else {
      // The last of the CTAs that share the row tile adds them up, in CTA order.
      if (warp == 0) {
        float* dst = p.part + static_cast<size_t>(s.slot) * C::kSlot;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int r = 8 * nt + 2 * t + h;
#pragma unroll
            for (int q = 0; q < WB; q += 2)
              __stcg(reinterpret_cast<float4*>(dst) + ((nt * 2 + h) * (WB / 2) + q / 2) * 32 + lane,
                     make_float4(o[q][nt][h], o[q][nt][h + 2], o[q + 1][nt][h], o[q + 1][nt][h + 2]));
            if (g == 0) __stcg(reinterpret_cast<float2*>(dst + ROWS * D) + r, make_float2(m[nt][h], l[nt][h]));
          }
        __syncwarp();
        if (lane == 0) {
          fence_acq_rel_gpu();
          const int done = atomicAdd(&p.cnt[s.cf], 1);
          *s_last = done == s.cl - s.cf;
          if (*s_last) {
            fence_acq_rel_gpu();
            p.cnt[s.cf] = 0;
          }
        }
      }
      __syncthreads();
      if (*s_last && s.cl - s.cf < kDirect) {
        // A thread has four elements of a row and loads all partials at once: their
        // latency is all that is left of the call by then.
        const int at = tid / 32, h = at / (WB / 2);   // (warp `at` has vector at % (WB / 2) of row 2t + (h & 1) of tile h / 2)
        const int jr = 8 * (h >> 1) + 2 * t + (h & 1), jc = g * (D / 8) + 4 * (at % (WB / 2)), r = s.r * ROWS + jr;
        if (jr < ROWS && r < rows) {
          float2 ml[kDirect];
          float4 v[kDirect];
#pragma unroll
          for (int i = 0; i < kDirect; ++i) {
            const int c = s.cf + i;
            if (c <= s.cl) {
              const float* src = p.part + static_cast<size_t>(2 * c + (i == 0 ? 1 : 0)) * C::kSlot;
              ml[i] = __ldcg(reinterpret_cast<const float2*>(src + ROWS * D) + jr);
              v[i] = __ldcg(reinterpret_cast<const float4*>(src) + tid);
            } else {
              ml[i] = make_float2(kNone, 0.f), v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            }
          }
          float mx = kNone, sum = 0.f, a[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int i = 0; i < kDirect; ++i) mx = fmaxf(mx, ml[i].x);
#pragma unroll
          for (int i = 0; i < kDirect; ++i) {
            const float w = exp2_approx(ml[i].x - mx);
            sum = fmaf(ml[i].y, w, sum);
            a[0] = fmaf(v[i].x, w, a[0]), a[1] = fmaf(v[i].y, w, a[1]);
            a[2] = fmaf(v[i].z, w, a[2]), a[3] = fmaf(v[i].w, w, a[3]);
          }
          const int tok = r / p.group, hd = s.h * p.group + (r - tok * p.group);
          const int64_t tk = s.start + tok;
          const float inv = sum == 0.f ? 0.f : 1.f / sum;   // 0: no token (a NaN is not)
          const __nv_bfloat162 z0 = __floats2bfloat162_rn(a[0] * inv, a[1] * inv), z1 = __floats2bfloat162_rn(a[2] * inv, a[3] * inv);
          *reinterpret_cast<uint2*>(p.out + tk * p.os + static_cast<int64_t>(hd) * D + jc) =
              make_uint2(*reinterpret_cast<const uint32_t*>(&z0), *reinterpret_cast<const uint32_t*>(&z1));
          if (jc == 0 && p.lse) p.lse[tk * p.Hq + hd] = sum == 0.f ? -INFINITY : (mx + log2f(sum)) * kLn2;
        }
      } else if (*s_last) {
        // warp k takes every eighth partial, then the warps are joined as above
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            m[nt][h] = kNone, l[nt][h] = 0.f;
#pragma unroll
            for (int q = 0; q < WB; ++q) o[q][nt][h] = 0.f, o[q][nt][h + 2] = 0.f;
          }
#pragma unroll 1
        for (int cc = s.cf + warp; cc <= s.cl; cc += kWarps) {
          const float* src = p.part + static_cast<size_t>(2 * cc + (cc == s.cf ? 1 : 0)) * C::kSlot;
          float4 v[NT][2][WB / 2];
          float2 other[NT][2];
          float f[NT][2], fo[NT][2];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int r = 8 * nt + 2 * t + h;
#pragma unroll
              for (int q = 0; q < WB / 2; ++q) v[nt][h][q] = __ldcg(reinterpret_cast<const float4*>(src) + ((nt * 2 + h) * (WB / 2) + q) * 32 + lane);
              other[nt][h] = __ldcg(reinterpret_cast<const float2*>(src + ROWS * D) + r);
            }
          merge(f, fo, other);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int q = 0; q < WB / 2; ++q) {
                const float4 x = v[nt][h][q];
                o[2 * q][nt][h] = fmaf(o[2 * q][nt][h], f[nt][h], x.x * fo[nt][h]);
                o[2 * q][nt][h + 2] = fmaf(o[2 * q][nt][h + 2], f[nt][h], x.y * fo[nt][h]);
                o[2 * q + 1][nt][h] = fmaf(o[2 * q + 1][nt][h], f[nt][h], x.z * fo[nt][h]);
                o[2 * q + 1][nt][h + 2] = fmaf(o[2 * q + 1][nt][h + 2], f[nt][h], x.w * fo[nt][h]);
              }
        }
        join();
        if (warp == 0) output();
      }
    }
    __syncthreads();   // the segment after the next is known, and nobody reads this one any more
    seg_ids = page_at(segs[(seg + 2) % 3], lane);
    if (on == seg) ++on;   // (after a wait that ran out)
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
  return flh::launch_early(k_kv8_rows<FMT, D, NT>, C::kCtas * flh::sm_count(), kRowsThreads, C::kSmem, s, km, vm, p);
}

template <int FMT, int D>
int pick_rows(const CUtensorMap& km, const CUtensorMap& vm, const AttnParams& p, long long rows, cudaStream_t s) {
  // Heads of 64 with more than 8 rows take tiles of 16 (16 sequences of 2 to 5
  // rows x 3 heads, 37 to 4001 tokens: 29 us against 31 us with tiles of 8; 64
  // rows over 4096 tokens: 87 against 117).  Heads of 128 always take tiles of 8:
  // the accumulators of 16 rows leave one CTA on an SM (12 rows: 44 us against
  // 36 us; 16 rows over 4096 tokens: 52 against 54).
  if constexpr (D == 64) {
    if (rows > 8) return launch_rows<FMT, D, 2>(km, vm, p, s);
  }
  return launch_rows<FMT, D, 1>(km, vm, p, s);
}

// What a call of T rows in B sequences, at most max_q of one sequence, launches,
// and the scratch of those kernels.  max_q may be loose: no sequence has more
// rows than T.  The size query, which knows no max_q, asks for T: the scratch
// does not fall with max_q, so its answer covers every call of these T and B.
struct AttnPlan {
  long long rows;      // most rows of a sequence, query heads of a kv head x tokens
  bool prompt, few;    // the kernels for many rows and for few
  size_t scratch;
};
AttnPlan attn_plan(int T, int B, int max_q, int group, int head_dim) {
  AttnPlan a;
  a.rows = static_cast<long long>(max_q < T ? max_q : T) * group;
  a.prompt = a.rows > kFewRows;
  a.few = !a.prompt || B > 1;   // one sequence goes to the one kernel; a batch may hold both kinds
  // two partials a CTA: the rows that it shares with the CTAs before and after
  const size_t few = 2ull * flh::sm_count() * 2 * 16 * (head_dim + 2) * 4;   // (two CTAs an SM)
  const size_t many = prompt_scratch(head_dim);
  a.scratch = a.prompt && many > few ? many : few;
  return a;
}

// Whether a row of `width` elements of `out` lies over one of q: CTAs read q's
// rows at any time of the call.  Rows of the two may alternate in one buffer.
bool rows_overlap(const void* q, int64_t qs, const void* out, int64_t os, int64_t width, int T) {
  const int64_t d = (reinterpret_cast<intptr_t>(out) - reinterpret_cast<intptr_t>(q)) / 2;   // elements; both are aligned
  if (d > -width && d < width) return true;
  if (qs != os || T == 1) return false;
  const int64_t rest = (d % qs + qs) % qs;   // from the row of q at or before a row of out
  return (rest < width || qs - rest < width) && d > -(T - 1) * qs - width && d < (T - 1) * qs + width;
}

}  // namespace

extern "C" int fl_kv8_attention_workspace(int T, int B, int Hq, int kv_heads, int head_dim, size_t* out) {
  if (!out || T < 1 || B < 1 || Hq < 1 || kv_heads < 1 || Hq % kv_heads) return FL_ERR_ARG;
  if (head_dim != 64 && head_dim != 128) return FL_ERR_UNSUPPORTED;
  *out = kScratchOff + attn_plan(T, B, T, Hq / kv_heads, head_dim).scratch;
  return FL_OK;
}

extern "C" int fl_kv8_test_plan(int T, int B, int max_q, int Hq, int kv_heads, int head_dim, long long* out) {
  if (!out || T < 1 || B < 1 || max_q < 1 || Hq < 1 || kv_heads < 1 || Hq % kv_heads || (head_dim != 64 && head_dim != 128))
    return FL_ERR_ARG;
  const AttnPlan a = attn_plan(T, B, max_q, Hq / kv_heads, head_dim);
  out[0] = a.rows, out[1] = a.prompt, out[2] = a.few, out[3] = static_cast<long long>(kScratchOff + a.scratch);
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
  if (rows_overlap(q, q_stride, out, out_stride, width, seqs->T)) return FL_ERR_ARG;
  const AttnPlan plan = attn_plan(seqs->T, seqs->B, seqs->max_q, Hq / cache->kv_heads, cache->head_dim);
  if (plan.rows > 0x7fffffffll) return FL_ERR_UNSUPPORTED;
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
  p.seqs = flh::seqs_of(*seqs);
  p.num_blocks = cache->num_blocks, p.block = cache->block, p.heads = cache->kv_heads;
  p.group = Hq / cache->kv_heads, p.Hq = Hq, p.window = window;
  p.scale2 = scale * 1.44269504088896340736f;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (plan.prompt) {
    if (!code_map(&km, cache->k, *cache, cache->block) || !code_map(&vm, cache->v, *cache, cache->block)) return FL_ERR_CUDA;
    p.rows_lo = plan.few ? kFewRows : 0, p.rows_hi = 0x7fffffff;
    const int e = launch_prompt(km, vm, p, cache->format, cache->head_dim, s);
    if (e != FL_OK || !plan.few) return e;
  }
  if (!code_map(&km, cache->k, *cache, 16) || !code_map(&vm, cache->v, *cache, 16)) return FL_ERR_CUDA;
  p.rows_lo = 0, p.rows_hi = kFewRows;
  if (cache->format == FL_KV8_E4M3)
    return cache->head_dim == 64 ? pick_rows<FL_KV8_E4M3, 64>(km, vm, p, plan.rows, s)
                                 : pick_rows<FL_KV8_E4M3, 128>(km, vm, p, plan.rows, s);
  return cache->head_dim == 64 ? pick_rows<FL_KV8_INT8, 64>(km, vm, p, plan.rows, s)
                               : pick_rows<FL_KV8_INT8, 128>(km, vm, p, plan.rows, s);
}
