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
// Inside a CTA a producer warp copies the units' pages by TMA (swizzled, so
// that both operand reads below are free of bank conflicts) into a ring, and
// eight warps take 16 tokens of each unit with a softmax state of their own,
// joined once a segment.  A warp's products are transposed, so that tokens
// fill the 16 rows of mma.sync and query rows its 8 columns:
//   S^T [16 tokens x 8 rows] = K q^T,   O^T [D x 8 rows] += V^T p^T.
// Codes become f16 in registers, exactly; the contraction index of either
// product may be permuted, so a lane reads 16 contiguous bytes: of its token's
// key for the first product, and of 4 tokens' values for the second, whose
// 4 x 4 bytes it transposes with byte permutes.
// Scales stay out of the operands.  q is brought to [1, 2) by a power of two a
// row (then f16 holds it with no loss that matters: 2^-25 of the row's largest
// value).  x is scaled in fp32.  p is rounded to f16 (2^-11, against the
// output's 2^-9) after a factor 2^14 v_scale / v_ref, v_ref the largest value
// scale so far, so that it keeps its 11 bits down to 2^-28 of the largest
// weight; the accumulators are in units of v_ref.  Sums are fp32.
#include "fl_kv8_prompt.cuh"
#include "fl_tc.cuh"

using namespace flkv;

namespace {

constexpr int kTile = 128;              // tokens of a unit
constexpr int kWarps = 8;               // consumer warps
constexpr int kRowsThreads = 32 * (kWarps + 1);
constexpr float kPScale = 16384.f;      // 2^14
// Most rows of a sequence (query heads of a kv head x tokens) that this kernel
// takes; sequences with more go to the tcgen05 kernel, in the same call.
constexpr int kFewRows = 64;

template <int D, int NT>
struct RowsCfg {
  static constexpr int kRows = 8 * NT;
  static constexpr int kHalf = kTile * D;            // keys (or values) of a stage
  static constexpr int kStage = 2 * kHalf;
  static constexpr int kStages = D == 128 ? (NT == 1 ? 5 : 4) : 8;
  static constexpr int kCombLd = D + 4;              // joined rows: conflict-free float2 writes
  static constexpr int kCombOff = kStages * kStage;
  static constexpr int kMlOff = kCombOff + kWarps * kRows * kCombLd * 4;
  static constexpr int kMetaOff = kMlOff + kWarps * kRows * 2 * 4;
  static constexpr int kBarOff = kMetaOff + kStages * kTile / 16 * 2 * 4;
  static constexpr int kSmem = kBarOff + 2 * kStages * 8 + 1024;
  static_assert(kSmem <= 232448, "shared memory");
  static constexpr int kSlot = kRows * (D + 2);      // floats of a partial: O, m, l
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
__global__ void __launch_bounds__(kRowsThreads, 1)
    k_kv8_rows(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap, const AttnParams p) {
  using C = RowsCfg<D, NT>;
  constexpr int ROWS = C::kRows, NS = C::kStages, KS = D / 16, WB = D / 16;   // WB: words of a lane's keys, m tiles of O^T
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* comb = reinterpret_cast<float*>(smem + C::kCombOff);
  float* ml = reinterpret_cast<float*>(smem + C::kMlOff);          // [warp][row][m, l]
  float2* meta = reinterpret_cast<float2*>(smem + C::kMetaOff);    // [stage][16 tokens]: key, value scale
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBarOff);
  uint64_t* empty = full + NS;
  __shared__ int s_last;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], kWarps);
    }
    fence_mbar_init();
  }

  __shared__ long long scratch[kRowsThreads / 32 + 2];
  const Start start = find_start<kRowsThreads>(scratch, p.seqs.B, blockIdx.x, gridDim.x, 1, [&](int b) { return seq_work<ROWS>(p, b).units; });
  const long long U = start.U;
  const int P = start.P, c = blockIdx.x;
  if (c >= P) return;
  Walk<ROWS> walk;
  walk.u = unit_begin(c, U, P);
  walk.end = unit_begin(c + 1, U, P);
  walk.b = start.b;
  walk.base = start.base;
  walk.w = seq_work<ROWS>(p, walk.b);
  const long long ubeg = walk.u;

  if (warp == kWarps) {
    // ---------------- producer: lane i has page i of a batch of 32 pages
    const int ppt = kTile / p.block, tiles = 32 / ppt, pbytes = p.block * D;
    int j = 0;
    bool ok = true;
    Segment s;
    while (ok && walk.next(p, s)) {
      const PageRun run = read_pages(walk.w.q, p.block, p.window);
      const int pg0 = (walk.w.t0 + s.t) * ppt;
      auto page_at = [&](int i) {   // page i of the segment, -1 for none
        const int pg = pg0 + i;
        if (i >= s.n * ppt || pg < run.first || pg >= run.first + run.n) return -1;
        const int id = page_block(p.seqs, s.b, pg, p.num_blocks);
        if (id < 0) set_status(p.status, FL_ERR_DEVICE_CHECK, 52);
        return id;
      };
      auto scales_of = [&](int id) {
        if (id < 0) return make_float2(1.f, 1.f);
        const int64_t at = static_cast<int64_t>(id) * p.heads + s.h;
        return make_float2(p.ks[at], p.vs[at]);
      };
      // page numbers are read two batches ahead, scales one
      int id0 = -1, id1 = page_at(lane), id2 = page_at(32 + lane);
      float2 sc0 = make_float2(1.f, 1.f), sc1 = sc0;
      bool have1 = false;
      for (int i = 0; i < s.n; ++i, ++j) {
        const int k = i % tiles;
        if (k == 0) {
          id0 = id1;
          id1 = id2;
          id2 = page_at((i / tiles + 2) * 32 + lane);
        }
        const int st = j % NS;
        if (j >= NS && !mbar_wait(&empty[st], static_cast<uint32_t>(j / NS - 1) & 1u)) {
          if (lane == 0) set_status(p.status, FL_ERR_TIMEOUT, 53);
          ok = false;
          break;
        }
        const bool mine = lane >= k * ppt && lane < (k + 1) * ppt;   // lanes with a page of this tile
        const uint32_t valid = __ballot_sync(0xffffffffu, mine && id0 >= 0);
        if (lane == 0 && valid) mbar_expect_tx(&full[st], 2u * pbytes * __popc(valid));
        __syncwarp();
        if (mine && id0 >= 0) {
          const int row = static_cast<int>((static_cast<int64_t>(id0) * p.heads + s.h) * p.block);
          uint8_t* dst = smem + st * C::kStage + (lane - k * ppt) * pbytes;
          tma_load_2d(dst, &kmap, 0, row, &full[st]);
          tma_load_2d(dst + C::kHalf, &vmap, 0, row, &full[st]);
        }
        if (k == 0) {
          sc0 = have1 ? sc1 : scales_of(id0);
          sc1 = scales_of(id1);
          have1 = true;
        }
        // slice l (16 tokens) takes the scales of the page that it lies in
        const int from = k * ppt + (lane & 7) * 16 / p.block;
        const float a = __shfl_sync(0xffffffffu, sc0.x, from), v = __shfl_sync(0xffffffffu, sc0.y, from);
        if (lane < kTile / 16) meta[st * (kTile / 16) + lane] = make_float2(a, v);
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[st]);
      }
    }
    if (!ok)   // let the copies in flight land before the CTA can exit
      for (int jj = j > NS ? j - NS : 0; jj < j; ++jj) mbar_wait(&full[jj % NS], static_cast<uint32_t>(jj / NS) & 1u);
    return;
  }

  // ------------------ consumers
  const int g = lane >> 2, t = lane & 3;
  bool ok = true;
  int j = 0;
  Segment s;
  while (walk.next(p, s)) {
    const SeqWork& w = walk.w;
    const int past = w.q.kv - w.q.n;   // position of the sequence's first row
    // query rows as the B operand: lane (g, t) has row g's elements [t D/4, (t+1) D/4)
    uint32_t qf[NT][KS][2];
    float fac[NT][2];
    int lim[NT][2];
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
      const uint32_t* a = &raw[0].x;
      uint32_t top = 0;   // the largest magnitude's bits
#pragma unroll
      for (int i = 0; i < D / 8; ++i) top = max(top, max(a[i] & 0x7fffu, (a[i] >> 16) & 0x7fffu));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int e = row_exponent(top);
      const float down = pow2i(-e);
#pragma unroll
      for (int i = 0; i < KS; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t v = a[2 * i + h];
          qf[nt][i][h] = pack_f16(__uint_as_float(v << 16) * down, __uint_as_float(v & 0xffff0000u) * down);
        }
      const float f = p.scale2 * pow2i(e);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        fac[nt][h] = __shfl_sync(0xffffffffu, f, 4 * (2 * t + h));
        const int rr = min(s.r * ROWS + 8 * nt + 2 * t + h, w.rows - 1);
        lim[nt][h] = past + rr / p.group + 1;
      }
    }
    // tokens that any, and that every row of the tile sees
    const int lim_lo = past + s.r * ROWS / p.group + 1;
    const int lim_hi = past + min(s.r * ROWS + ROWS - 1, w.rows - 1) / p.group + 1;
    const int low_lo = p.window ? lim_lo - p.window : 0, low_hi = p.window ? lim_hi - p.window : 0;

    float o[WB][NT][4];
    float m[NT][2], l[NT][2], vref = 0.f;
#pragma unroll
    for (int i = 0; i < WB; ++i)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[i][nt][k] = 0.f;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int h = 0; h < 2; ++h) m[nt][h] = -INFINITY, l[nt][h] = 0.f;

    for (int i = 0; i < s.n; ++i, ++j) {
      const int st = j % NS;
      if (ok && !mbar_wait(&full[st], static_cast<uint32_t>(j / NS) & 1u)) {
        if (lane == 0) set_status(p.status, FL_ERR_TIMEOUT, 54);
        ok = false;   // no more waits: the rest is walked through without data
      }
      const int pos = (w.t0 + s.t + i) * kTile + 16 * warp;   // the warp's first token
      if (ok && pos < lim_hi && pos + 16 > low_lo) {
        const uint8_t* kt = smem + st * C::kStage + warp * 16 * D;
        const uint8_t* vt = kt + C::kHalf;
        const float2 sc = meta[st * (kTile / 16) + warp];
        // S^T = K q^T
        float x[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 4; ++k) x[nt][k] = 0.f;
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
            for (int nt = 0; nt < NT; ++nt) mma_f16(x[nt], a0, a1, a2, a3, qf[nt][k][0], qf[nt][k][1]);
          }
        }
        const bool mask = pos + 16 > lim_lo || pos < low_hi;
        bool grow = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            x[nt][k] *= sc.x * fac[nt][k & 1];
            if (mask) {
              const int tok = pos + g + (k >> 1) * 8;
              const int lm = lim[nt][k & 1];
              if (tok >= lm || (p.window && tok < lm - p.window)) x[nt][k] = -INFINITY;
            }
            grow |= x[nt][k] > m[nt][k & 1];
          }
        if (__any_sync(0xffffffffu, grow) || sc.y > vref) {
          // a larger maximum of some row, or a larger value scale
          const float vnew = fmaxf(vref, sc.y), vr = vref / vnew;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float mx = fmaxf(fmaxf(x[nt][h], x[nt][h + 2]), m[nt][h]);
              mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
              mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
              mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
              const float f = mx == -INFINITY ? 1.f : exp2_approx(m[nt][h] - mx);
              m[nt][h] = mx;
              l[nt][h] *= f;
#pragma unroll
              for (int q = 0; q < WB; ++q) {
                o[q][nt][h] *= f * vr;
                o[q][nt][h + 2] *= f * vr;
              }
            }
          vref = vnew;
        }
        const float pv = kPScale * (sc.y / vref);
        uint32_t pb[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float e[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float mm = m[nt][k & 1];
            e[k] = exp2_approx(x[nt][k] - (mm == -INFINITY ? 0.f : mm));
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
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[st]);
    }

    // ---------------- join the eight warps
    const float back = vref / kPScale;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float sum = l[nt][h];
        sum += __shfl_xor_sync(0xffffffffu, sum, 4);
        sum += __shfl_xor_sync(0xffffffffu, sum, 8);
        sum += __shfl_xor_sync(0xffffffffu, sum, 16);
        const int row = 8 * nt + 2 * t + h;
        if (g == 0) reinterpret_cast<float2*>(ml)[warp * ROWS + row] = make_float2(m[nt][h], sum);
        float* dst = comb + (warp * ROWS + row) * C::kCombLd + 2 * g;
#pragma unroll
        for (int i = 0; i < WB; ++i)
          *reinterpret_cast<float2*>(dst + 16 * i) = make_float2(o[i][nt][h] * back, o[i][nt][h + 2] * back);
      }
    named_bar(1, 32 * kWarps);
    const bool whole = s.n == w.nt;
    float* slot = p.part + static_cast<size_t>(2 * c + (s.first < ubeg ? 0 : 1)) * C::kSlot;
    for (int i = tid; i < ROWS * D / 2; i += 32 * kWarps) {
      const int row = i / (D / 2), d = 2 * (i - row * (D / 2));
      const int at = d % (D / 8) / 2 * 16 + d / (D / 8) * 2;
      float mx = -INFINITY;
#pragma unroll
      for (int k = 0; k < kWarps; ++k) mx = fmaxf(mx, ml[2 * (k * ROWS + row)]);
      float sum = 0.f, ox = 0.f, oy = 0.f;
#pragma unroll
      for (int k = 0; k < kWarps; ++k) {
        const float mk = ml[2 * (k * ROWS + row)];
        const float f = mk == -INFINITY ? 0.f : exp2_approx(mk - mx);
        const float2 v = *reinterpret_cast<const float2*>(comb + (k * ROWS + row) * C::kCombLd + at);
        sum = fmaf(f, ml[2 * (k * ROWS + row) + 1], sum);
        ox = fmaf(f, v.x, ox), oy = fmaf(f, v.y, oy);
      }
      if (!whole) {
        __stcg(reinterpret_cast<float2*>(slot + row * D + d), make_float2(ox, oy));
        if (d == 0) __stcg(reinterpret_cast<float2*>(slot + ROWS * D + 2 * row), make_float2(mx, sum));
        continue;
      }
      const int r = s.r * ROWS + row;
      if (r < w.rows) {
        const int tok = r / p.group, hd = s.h * p.group + (r - tok * p.group);
        const int64_t tk = w.q.start + tok;
        const float inv = sum == 0.f ? 0.f : 1.f / sum;   // 0: no token (a NaN is not)
        *reinterpret_cast<__nv_bfloat162*>(p.out + tk * p.os + static_cast<int64_t>(hd) * D + d) =
            __floats2bfloat162_rn(ox * inv, oy * inv);
        if (d == 0 && p.lse) p.lse[tk * p.Hq + hd] = sum == 0.f ? -INFINITY : (mx + log2f(sum)) * kLn2;
      }
    }
    if (!whole) {
      // the last of the CTAs that share the row tile adds them up, in CTA order
      const int cf = cta_of_unit(s.first, U, P), cl = cta_of_unit(s.first + w.nt - 1, U, P);
      named_bar(1, 32 * kWarps);
      if (tid == 0) {
        fence_acq_rel_gpu();
        const int done = atomicAdd(&p.cnt[cf], 1);
        s_last = done == cl - cf;
        if (s_last) {
          fence_acq_rel_gpu();
          p.cnt[cf] = 0;
        }
      }
      named_bar(1, 32 * kWarps);
      if (s_last) {
        auto slot_of = [&](int cc) {
          return p.part + static_cast<size_t>(2 * cc + (s.first < unit_begin(cc, U, P) ? 0 : 1)) * C::kSlot;
        };
        for (int i = tid; i < ROWS * D / 2; i += 32 * kWarps) {
          const int row = i / (D / 2), d = 2 * (i - row * (D / 2));
          const int r = s.r * ROWS + row;
          if (r >= w.rows) continue;
          float mx = -INFINITY;
          for (int cc = cf; cc <= cl; ++cc) mx = fmaxf(mx, __ldcg(slot_of(cc) + ROWS * D + 2 * row));
          float sum = 0.f, ox = 0.f, oy = 0.f;
          for (int cc = cf; cc <= cl; ++cc) {
            const float2 a = __ldcg(reinterpret_cast<const float2*>(slot_of(cc) + ROWS * D + 2 * row));
            const float2 v = __ldcg(reinterpret_cast<const float2*>(slot_of(cc) + row * D + d));
            const float f = a.x == -INFINITY ? 0.f : exp2_approx(a.x - mx);
            sum = fmaf(f, a.y, sum);
            ox = fmaf(f, v.x, ox), oy = fmaf(f, v.y, oy);
          }
          const int tok = r / p.group, hd = s.h * p.group + (r - tok * p.group);
          const int64_t tk = w.q.start + tok;
          const float inv = sum == 0.f ? 0.f : 1.f / sum;   // 0: no token (a NaN is not)
          *reinterpret_cast<__nv_bfloat162*>(p.out + tk * p.os + static_cast<int64_t>(hd) * D + d) =
              __floats2bfloat162_rn(ox * inv, oy * inv);
          if (d == 0 && p.lse) p.lse[tk * p.Hq + hd] = sum == 0.f ? -INFINITY : (mx + log2f(sum)) * kLn2;
        }
      }
    }
    named_bar(1, 32 * kWarps);   // the joined rows and s_last are read before the next segment writes them
  }
}

// ------------------------------------------------------------------ host
// The codes as rows of head_dim bytes, one page of one head a box.
bool code_map(CUtensorMap* map, void* base, const fl_kv8_cache& c) {
  auto enc = flh::encode_fn();
  if (!enc) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(c.head_dim),
                              static_cast<cuuint64_t>(c.num_blocks) * c.kv_heads * c.block};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(c.head_dim)};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(c.head_dim), static_cast<cuuint32_t>(c.block)};
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
  k_kv8_rows<FMT, D, NT><<<flh::sm_count(), kRowsThreads, C::kSmem, s>>>(km, vm, p);
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
  const size_t slot = prompt ? prompt_slot_floats(head_dim) : 16 * (head_dim + 2);
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
  if (!code_map(&km, cache->k, *cache) || !code_map(&vm, cache->v, *cache)) return FL_ERR_CUDA;
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
    // one sequence goes to the one kernel; a batch may hold both kinds
    p.rows_lo = seqs->B > 1 ? kFewRows : 0, p.rows_hi = 0x7fffffff;
    const int e = launch_prompt(km, vm, p, cache->format, cache->head_dim, s);
    if (e != FL_OK || seqs->B == 1) return e;
  }
  p.rows_lo = 0, p.rows_hi = kFewRows;
  if (cache->format == FL_KV8_E4M3)
    return cache->head_dim == 64 ? pick_rows<FL_KV8_E4M3, 64>(km, vm, p, rows, s)
                                 : pick_rows<FL_KV8_E4M3, 128>(km, vm, p, rows, s);
  return cache->head_dim == 64 ? pick_rows<FL_KV8_INT8, 64>(km, vm, p, rows, s)
                               : pick_rows<FL_KV8_INT8, 128>(km, vm, p, rows, s);
}
