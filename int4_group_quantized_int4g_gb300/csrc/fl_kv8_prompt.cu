// Attention over the 8-bit paged cache for many query rows (prompts, chunks):
// the contraction-bound form, on tcgen05.
//
// An item is 256 rows of a kv head (rows are (token, query head of the group),
// so that a group shares its keys) in two tiles of 128, a unit one item x 128
// tokens.  The units of the batch lie in one line and each of the persistent
// CTAs (one an SM) takes an equal run of them, so ragged batches, the causal
// triangle and few rows over a long context all fill the GPU; an item that
// several CTAs share is joined by the last of them, in CTA order.
//
// Per unit: S = Q K^T (128 x 128 a row tile, fp32 in tensor memory), softmax
// with the running maximum and sum, P as f16 back into S's columns, O += P V
// (P from tensor memory, O there too).  Codes become f16 once per CTA and unit,
// in shared memory, and serve both row tiles.  Warps:
//   0..3, 4..7  softmax of row tile 0, 1: a thread has a row.  The maximum
//               that weights are taken against moves only when it is passed by
//               2^8; then the warp rescales its rows of O in tensor memory
//   8..11       convert: key rows as they are (K-major), values transposed
//               (tokens along K) with byte permutes; the order of output
//               columns is free, so value element 4 l + j goes to row j D/4 + l,
//               which makes the writes conflict-free
//   12, 13      issue the MMAs of row tile 0, 1
//   14          copies pages by TMA into a staging tile for keys and for values
//
// Scales: with e_b the power of two in a block's scale and e_ref the largest of
// the sequence's head, codes are multiplied by 2^(e_b - e_ref + k) as they
// become f16 (exact down to 2^-24 of f16: blocks whose scales are 2^20 apart)
// and the reference goes into the row's factor or the output.  Mantissas of
// scales other than powers of two multiply S and P, for the sequences that have
// them.  q as in the kernel for few rows.  P is f16 (2^-11, the output's
// rounding is 2^-9) times 2^6, and up to 2^14; its fp32 sum is taken before.
#include "fl_kv8_prompt.cuh"
#include "fl_tc.cuh"

using namespace flkv;

namespace {

constexpr int kPrThreads = 512;
constexpr int kConv0 = 8, kIssue0 = 12, kProd = 14;   // first warps of the roles
constexpr float kBias = 6.f;                          // P = 2^(x - m + kBias)
constexpr float kSlack = 8.f;                         // the maximum may lag by 2^kSlack

template <int D>
struct PrCfg {
  static constexpr int kQ = 128 * D * 2;       // a row tile of q
  static constexpr int kKv = 128 * D * 2;      // keys or values of a unit as f16
  static constexpr int kStg = 128 * D;         // their codes
  static constexpr int kKOff = 2 * kQ;         // two stages
  static constexpr int kVOff = kKOff + 2 * kKv;
  static constexpr int kStgOff = kVOff + 2 * kKv;
  static constexpr int kMetaOff = kStgOff + 2 * kStg;      // [4 units][8 slices of 16 tokens]: key, value scale
  static constexpr int kRefOff = kMetaOff + 4 * 8 * 8;     // [4 segments]: exponents, general
  static constexpr int kBarOff = kRefOff + 4 * 16;
  static constexpr int kBars = 4 + 8 + 2 + 2 + 2 + 2 + 8;
  static constexpr int kSmem = kBarOff + kBars * 8 + 64 + 1024;
  static constexpr int kSlot = kPromptRows * (D + 2);      // floats of a partial: O [D][256], m, l [256][2]
  static_assert(kSmem <= 232448, "shared memory");
};

// f16 in, fp32 out, both K-major, M = 128
__device__ __forceinline__ uint32_t idesc_f16(int n) {
  return (1u << 4) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(128 >> 4) << 24);
}
__device__ __forceinline__ void umma_f16_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void umma_f16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void tmem_ld32_issue(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld32_wait(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                 "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_ld8_issue(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld8_wait(uint32_t (&r)[8]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

// A run of units of one item inside the CTA's units.
struct Seg {
  int b, h, item, t, n, nt;   // units [t, t + n) of the item's nt
  int tile0;                  // the item's first tile
  long long first;            // the item's first unit
};
struct PromptWalk {
  long long u, end, base;
  int b;
  PromptWork w;
  __device__ void load(const AttnParams& p) {
    w = prompt_work(seq_info(p.seqs, b, p.block), p.group, p.heads, p.window, p.rows_lo, p.rows_hi);
  }
  __device__ bool next(const AttnParams& p, Seg& s) {
    if (u >= end) return false;
    while (u >= base + w.per_head * p.heads) {
      base += w.per_head * p.heads;
      if (++b >= p.seqs.B) return false;
      load(p);
    }
    const long long local = u - base;
    s.b = b;
    s.h = static_cast<int>(local / w.per_head);
    const long long in_head = local - s.h * w.per_head;
    s.item = w.item_of(in_head);
    s.t = static_cast<int>(in_head - w.before(s.item));
    s.nt = w.tiles(s.item);
    s.n = static_cast<int>(min(static_cast<long long>(s.nt - s.t), end - u));
    s.tile0 = w.first_tile(s.item);
    s.first = u - s.t;
    u += s.n;
    return true;
  }
};
// Units of the segment in which row tile t (0 or 1) has a visible token; the
// CTA works through as many as the larger.
__device__ __forceinline__ int live_units(const PromptWork& w, const Seg& s, int t) {
  const int r0 = s.item * kPromptRows + 128 * t;
  if (r0 >= w.rows) return 0;
  return min(max((max(w.lim(r0, 128), 0) + kPromptTile - 1) / kPromptTile - s.tile0 - s.t, 0), s.n);
}

// A scale's power of two and what is left of it.
__device__ __forceinline__ int scale_exponent(float s) {
  return min(max(static_cast<int>((__float_as_uint(s) >> 23) & 255u) - 127, -126), 126);
}
__device__ __forceinline__ float scale_mantissa(float s) { return s * pow2i(-scale_exponent(s)); }

// codes' multiplier exponent: the largest code times 2^k is far inside f16,
// and for integers so is 1152 * 2^k
template <int FMT>
__device__ __forceinline__ constexpr int code_shift() {
  return FMT == FL_KV8_E4M3 ? 7 : 5;
}
// Two codes (low or high half of w) times r, as f16: (1024 + u) r - 1152 r for
// integers, one rounding.  r2: r twice; o2: -1152 r twice.
template <int FMT, bool HI>
__device__ __forceinline__ uint32_t scaled_pair(uint32_t w, __half2 r2, __half2 o2) {
  __half2 v;
  if constexpr (FMT == FL_KV8_E4M3) {
    const uint32_t c = code_pair_f16<FMT, HI>(w);
    v = __hmul2(*reinterpret_cast<const __half2*>(&c), r2);
  } else {
    const uint32_t u = __byte_perm(w, 0x64646464u, HI ? 0x4342u : 0x4140u);
    v = __hfma2(*reinterpret_cast<const __half2*>(&u), r2, o2);
  }
  return *reinterpret_cast<const uint32_t*>(&v);
}

template <int FMT, int D>
__global__ void __launch_bounds__(kPrThreads, 1)
    k_kv8_prompt(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap, const AttnParams p) {
  using C = PrCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float2* meta = reinterpret_cast<float2*>(smem + C::kMetaOff);
  int4* refs = reinterpret_cast<int4*>(smem + C::kRefOff);
  uint64_t* stg_full = reinterpret_cast<uint64_t*>(smem + C::kBarOff);   // [keys, values]
  uint64_t* stg_empty = stg_full + 2;
  uint64_t* k_full = stg_empty + 2;      // [stage]
  uint64_t* k_empty = k_full + 2;
  uint64_t* v_full = k_empty + 2;
  uint64_t* v_empty = v_full + 2;
  uint64_t* q_full = v_empty + 2;        // [row tile]
  uint64_t* s_full = q_full + 2;
  uint64_t* p_full = s_full + 2;
  uint64_t* o_done = p_full + 2;
  uint64_t* ref_full = o_done + 2;       // [4]
  uint64_t* ref_empty = ref_full + 4;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(ref_empty + 4);
  int* s_last = reinterpret_cast<int*>(tmem_slot + 1);
  int* s_red = s_last + 1;               // [converter warp][3]: largest exponents, whether there are mantissas

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&stg_full[i], 1);
      mbar_init(&stg_empty[i], 4);
      mbar_init(&k_full[i], 4);
      mbar_init(&k_empty[i], 2);
      mbar_init(&v_full[i], 4);
      mbar_init(&v_empty[i], 2);
      mbar_init(&q_full[i], 4);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
      mbar_init(&o_done[i], 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&ref_full[i], 1);
      mbar_init(&ref_empty[i], kConv0);
    }
    fence_mbar_init();
  }
  const Start start = find_start<kPrThreads>(p.seqs.B, 2, [&](int b) {
    return prompt_work(seq_info(p.seqs, b, p.block), p.group, p.heads, p.window, p.rows_lo, p.rows_hi).per_head * p.heads;
  });
  const long long U = start.U;
  const int P = start.P, c = blockIdx.x;
  if (c >= P) return;
  if (warp == kIssue0) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  cta_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;   // S/P of row tile t at 128 t, O at 256 + D t
  PromptWalk walk;
  walk.u = unit_begin(c, U, P);
  walk.end = unit_begin(c + 1, U, P);
  walk.b = start.b;
  walk.base = start.base;
  walk.load(p);
  const long long ubeg = walk.u;
  bool ok = true;   // false after a wait ran out: nothing is waited for or issued any more
  auto wait = [&](uint64_t* bar, uint32_t phase, int where) {
    if (ok && !mbar_wait(bar, phase & 1u)) {
      set_status(p.status, FL_ERR_TIMEOUT, where);
      ok = false;
    }
  };
  Seg s;

  if (warp < kConv0) {
    // ---------------- softmax and output: a thread has row r of row tile t
    const int t = warp >> 2, r = (warp & 3) * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lanes + 128 * t, to = tmem + lanes + 256 + D * t;
    uint32_t js = 0;    // units of this row tile so far
    int seg = 0;
    while (walk.next(p, s)) {
      const PromptWork& w = walk.w;
      const int r0 = s.item * kPromptRows + 128 * t, row = r0 + r;
      const int live = live_units(w, s, t);
      const bool real = row < w.rows;
      const int tok = min(row, w.rows - 1) / p.group;
      const int hd = s.h * p.group + (row - tok * p.group);   // (of a real row)
      const int64_t tk = static_cast<int64_t>(w.q.start) + tok;
      float a = 0.f;
      wait(&ref_full[seg & 3], seg >> 2, 60);
      const int4 ref = refs[seg & 3];   // exponents of keys and values, mantissas or not, the first unit's place in meta
      __syncwarp();
      if (lane == 0) mbar_arrive(&ref_empty[seg & 3]);
      ++seg;
      if (live > 0) {
        // the row of q, times a power of two and the sign of the scale, as f16
        uint4 x[D / 8];
#pragma unroll
        for (int i = 0; i < D / 8; ++i) x[i] = make_uint4(0, 0, 0, 0);
        if (real) {
          const uint4* src = reinterpret_cast<const uint4*>(p.q + tk * p.qs + static_cast<int64_t>(hd) * D);
#pragma unroll
          for (int i = 0; i < D / 8; ++i) x[i] = src[i];
        }
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          const uint32_t v[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
          for (int k = 0; k < 4; ++k) top = max(top, max(v[k] & 0x7fffu, (v[k] >> 16) & 0x7fffu));
        }
        const int e = row_exponent(top);
        const float down = copysignf(pow2i(-e), p.scale2);
        a = fabsf(p.scale2) * pow2i(e) * pow2i(max(ref.x - code_shift<FMT>(), -126));
        uint8_t* q = smem + t * C::kQ + r * 128;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          const uint32_t v[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
          uint32_t o[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            o[k] = pack_f16(__uint_as_float(v[k] << 16) * down, __uint_as_float(v[k] & 0xffff0000u) * down);
          *reinterpret_cast<uint4*>(q + (i >> 3) * (128 * 128) + (((i & 7) ^ (r & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_full[t]);
      }
      const int lim = w.past + tok + 1, low = w.window ? lim - w.window : 0;      // tokens [low, lim) of this row
      const int lim_lo = w.past + r0 / p.group + 1;                               // of all rows of the tile
      const int low_hi = w.window ? w.lim(r0, 128) - w.window : 0;
      float m = -INFINITY, l = 0.f;   // weights are 2^(x - m); m is kBias below the maximum that it was taken from
      for (int j = 0; j < live; ++j, ++js) {
        const int pos = (s.tile0 + s.t + j) * kPromptTile;
        const bool mask = pos + kPromptTile > lim_lo || pos < low_hi;
        wait(&s_full[t], js, 61);
        tc_fence_after();
        uint32_t u[2][32];
        auto value = [&](uint32_t bits, int col, float mk) {   // x of a column
          float x = __uint_as_float(bits);
          if (ref.z) x *= mk;
          if (mask && (pos + col >= lim || pos + col < low)) x = -INFINITY;
          return x;
        };
        float mx = -INFINITY;
        tmem_ld32_issue(ts, u[0]);
        tmem_ld32_wait(u[0]);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (k < 3) tmem_ld32_issue(ts + 32 * (k + 1), u[(k + 1) & 1]);
          float m2[2] = {1.f, 1.f};
          if (ref.z) {
            m2[0] = scale_mantissa(meta[((ref.w + j) & 3) * 8 + 2 * k].x);
            m2[1] = scale_mantissa(meta[((ref.w + j) & 3) * 8 + 2 * k + 1].x);
          }
          if (!mask && !ref.z) {
#pragma unroll
            for (int i = 0; i < 32; ++i) mx = fmaxf(mx, __uint_as_float(u[k & 1][i]));
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) mx = fmaxf(mx, value(u[k & 1][i], 32 * k + i, m2[i >> 4]));
          }
          if (k < 3) tmem_ld32_wait(u[(k + 1) & 1]);
        }
        const float top = mx == -INFINITY ? -INFINITY : mx * a;   // (a may be 0)
        if (j == 0) {
          m = top - kBias;
        } else if (__any_sync(0xffffffffu, top - kBias > m + kSlack)) {
          // a maximum has outgrown its reference: the warp's rows of O move
          float f = 1.f;
          if (top - kBias > m + kSlack) {
            f = exp2_approx(m - (top - kBias));
            m = top - kBias;
          }
          l *= f;
          wait(&o_done[t], js - 1, 62);
          tc_fence_after();
#pragma unroll
          for (int k = 0; k < D / 32; ++k) {
            uint32_t o[32];
            tmem_ld32_issue(to + 32 * k, o);
            tmem_ld32_wait(o);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
            tmem_st32(to + 32 * k, o);
          }
          tmem_wait_st();
        }
        const float mm = m == -INFINITY ? 0.f : m;
        tmem_ld32_issue(ts, u[0]);
        tmem_ld32_wait(u[0]);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (k < 3) tmem_ld32_issue(ts + 32 * (k + 1), u[(k + 1) & 1]);
          uint32_t pk[16];
          if (!mask && !ref.z) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float e0 = exp2_approx(fmaf(__uint_as_float(u[k & 1][2 * i]), a, -mm));
              const float e1 = exp2_approx(fmaf(__uint_as_float(u[k & 1][2 * i + 1]), a, -mm));
              l += e0 + e1;
              pk[i] = pack_f16(e0, e1);
            }
          } else {
            float m2[2] = {1.f, 1.f}, n2[2] = {1.f, 1.f};
            if (ref.z) {
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const float2 sc = meta[((ref.w + j) & 3) * 8 + 2 * k + h];
                m2[h] = scale_mantissa(sc.x), n2[h] = scale_mantissa(sc.y);
              }
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              // (-inf * 0 of a masked column would be NaN: a is not applied to it)
              const float x0 = value(u[k & 1][2 * i], 32 * k + 2 * i, m2[i >> 3]);
              const float x1 = value(u[k & 1][2 * i + 1], 32 * k + 2 * i + 1, m2[i >> 3]);
              const float e0 = x0 == -INFINITY ? 0.f : exp2_approx(fmaf(x0, a, -mm));
              const float e1 = x1 == -INFINITY ? 0.f : exp2_approx(fmaf(x1, a, -mm));
              l += e0 + e1;
              pk[i] = pack_f16(e0 * n2[i >> 3], e1 * n2[i >> 3]);
            }
          }
          // P's columns 16 k .. lie over S's that have been read
          if (k < 3) tmem_ld32_wait(u[(k + 1) & 1]);
          tmem_st16(ts + 16 * k, pk);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[t]);
      }

      // ---------------- the rows' output, or their partial
      if (live > 0) {
        wait(&o_done[t], js - 1, 63);
        tc_fence_after();
      }
      const bool whole = s.n == s.nt;
      const float back = pow2i(max(ref.y - code_shift<FMT>(), -126));
      float* slot = p.part + static_cast<size_t>(2 * c + (s.first < ubeg ? 0 : 1)) * C::kSlot;
      const int slot_row = 128 * t + r;
      if (whole) {
        const float inv = l == 0.f ? 0.f : back / l;   // 0: no token (a NaN is not)
        __nv_bfloat16* dst = p.out + tk * p.os + static_cast<int64_t>(hd) * D;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          // elements 32 i .. 32 i + 31: columns 8 i .. 8 i + 7 of each quarter
          uint32_t o[4][8];
          if (live > 0) {
#pragma unroll
            for (int q = 0; q < 4; ++q) tmem_ld8_issue(to + q * (D / 4) + 8 * i, o[q]);
#pragma unroll
            for (int q = 0; q < 4; ++q) tmem_ld8_wait(o[q]);
          }
          if (real) {
            uint32_t v[16];
#pragma unroll
            for (int k = 0; k < 8; ++k)
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                const float x = live > 0 ? __uint_as_float(o[2 * q][k]) * inv : 0.f;
                const float y = live > 0 ? __uint_as_float(o[2 * q + 1][k]) * inv : 0.f;
                const __nv_bfloat162 z = __floats2bfloat162_rn(x, y);
                v[2 * k + q] = *reinterpret_cast<const uint32_t*>(&z);
              }
#pragma unroll
            for (int k = 0; k < 4; ++k)
              *reinterpret_cast<uint4*>(dst + 32 * i + 8 * k) = make_uint4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
          }
        }
        if (real && p.lse) p.lse[tk * p.Hq + hd] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
        continue;
      }
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        uint32_t o[32];
        if (live > 0) {
          tmem_ld32_issue(to + 32 * i, o);
          tmem_ld32_wait(o);
        }
#pragma unroll
        for (int k = 0; k < 32; ++k)
          __stcg(slot + (32 * i + k) * kPromptRows + slot_row, live > 0 ? __uint_as_float(o[k]) * back : 0.f);
      }
      __stcg(reinterpret_cast<float2*>(slot + D * kPromptRows) + slot_row, make_float2(m, l));
      // the last of the CTAs that share the item adds them up, in CTA order
      const int cf = cta_of_unit(s.first, U, P), cl = cta_of_unit(s.first + s.nt - 1, U, P);
      named_bar(1, 256);
      if (tid == 0) {
        fence_acq_rel_gpu();
        const int done = atomicAdd(&p.cnt[cf], 1);
        *s_last = done == cl - cf;
        if (*s_last) {
          fence_acq_rel_gpu();
          p.cnt[cf] = 0;
        }
      }
      named_bar(1, 256);
      const bool last = *reinterpret_cast<volatile int*>(s_last);
      named_bar(1, 256);   // (read before the next shared item's ticket)
      if (!last || !real) continue;
      auto slot_of = [&](int cc) {
        return p.part + static_cast<size_t>(2 * cc + (s.first < unit_begin(cc, U, P) ? 0 : 1)) * C::kSlot;
      };
      float mx = -INFINITY;
      for (int cc = cf; cc <= cl; ++cc) mx = fmaxf(mx, __ldcg(slot_of(cc) + D * kPromptRows + 2 * slot_row));
      float sum = 0.f;
      for (int cc = cf; cc <= cl; ++cc) {
        const float2 v = __ldcg(reinterpret_cast<const float2*>(slot_of(cc) + D * kPromptRows) + slot_row);
        sum = fmaf(v.x == -INFINITY ? 0.f : exp2_approx(v.x - mx), v.y, sum);
      }
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      __nv_bfloat16* dst = p.out + tk * p.os + static_cast<int64_t>(hd) * D;
#pragma unroll 1
      for (int i = 0; i < D / 32; ++i) {
        float o[32];
#pragma unroll
        for (int k = 0; k < 32; ++k) o[k] = 0.f;
        for (int cc = cf; cc <= cl; ++cc) {
          const float* sl = slot_of(cc);
          const float mv = __ldcg(sl + D * kPromptRows + 2 * slot_row);
          const float f = mv == -INFINITY ? 0.f : exp2_approx(mv - mx);
#pragma unroll
          for (int k = 0; k < 32; ++k)   // element 32 i + k lies in column (k % 4) D/4 + 8 i + k / 4
            o[k] = fmaf(f, __ldcg(sl + ((k & 3) * (D / 4) + 8 * i + (k >> 2)) * kPromptRows + slot_row), o[k]);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t v[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const __nv_bfloat162 z = __floats2bfloat162_rn(o[8 * k + 2 * q] * inv, o[8 * k + 2 * q + 1] * inv);
            v[q] = *reinterpret_cast<const uint32_t*>(&z);
          }
          *reinterpret_cast<uint4*>(dst + 32 * i + 8 * k) = make_uint4(v[0], v[1], v[2], v[3]);
        }
      }
      if (p.lse) p.lse[tk * p.Hq + hd] = sum == 0.f ? -INFINITY : (mx + log2f(sum)) * kLn2;
    }
  } else if (warp < kIssue0) {
    // ---------------- convert
    const int ct = tid - 32 * kConv0, cw = warp - kConv0;
    int i = 0, seg = 0;
    int ref_b = -1, ref_h = -1, ke = -126, ve = -126, general = 0;
    while (walk.next(p, s)) {
      const PromptWork& w = walk.w;
      const int units = max(live_units(w, s, 0), live_units(w, s, 1));
      if (s.b != ref_b || s.h != ref_h) {
        // the largest powers of two of the scales of every page that a row sees
        ref_b = s.b, ref_h = s.h;
        const PageRun run = read_pages(w.q, p.block, p.window);
        ke = ve = -126;
        general = 0;
        for (int pg = ct; pg < run.n; pg += 128) {
          const int id = page_block(p.seqs, s.b, run.first + pg, p.num_blocks);
          if (id < 0) continue;
          const int64_t at = static_cast<int64_t>(id) * p.heads + s.h;
          const float a = p.ks[at], b = p.vs[at];
          ke = max(ke, scale_exponent(a)), ve = max(ve, scale_exponent(b));
          general |= scale_mantissa(a) != 1.f || scale_mantissa(b) != 1.f;
        }
        ke = __reduce_max_sync(0xffffffffu, ke);
        ve = __reduce_max_sync(0xffffffffu, ve);
        general = __any_sync(0xffffffffu, general);
        if (lane == 0) s_red[3 * cw] = ke, s_red[3 * cw + 1] = ve, s_red[3 * cw + 2] = general;
        named_bar(2, 128);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          ke = max(ke, s_red[3 * k]), ve = max(ve, s_red[3 * k + 1]);
          general |= s_red[3 * k + 2];
        }
        named_bar(2, 128);   // (read before the next head's)
      }
      wait(&ref_empty[seg & 3], (seg >> 2) + 1, 74);
      if (ct == 0) {
        refs[seg & 3] = make_int4(ke, ve, general, i & 3);
        mbar_arrive(&ref_full[seg & 3]);
      }
      ++seg;
      const int seen = first_seen(w.q, p.window);
      for (int j = 0; j < units; ++j, ++i) {
        const int st = i & 1;
        const float2* mt = meta + (i & 3) * 8;
        // 2^(e - e_ref + shift), 0 below f16 (pages that are not read have a scale of 1, which may exceed e_ref)
        auto ratio = [&](float scale, int e_ref) {
          return __float2half2_rn(pow2i(max(min(scale_exponent(scale) - e_ref, 0) + code_shift<FMT>(), -126)));
        };
        // keys
        wait(&stg_full[0], i, 64);
        wait(&k_empty[st], (i >> 1) + 1, 65);
        {
          const uint8_t* src = smem + C::kStgOff;
          uint8_t* dst = smem + C::kKOff + st * C::kKv;
          constexpr int kCh = D / 16, kIt = kCh;   // chunks of 16 codes a row, passes
#pragma unroll
          for (int it = 0; it < kIt; ++it) {
            const int task = it * 128 + ct, row = task / kCh, ch = task % kCh;
            const __half2 r2 = ratio(mt[row >> 4].x, ke), o2 = __hmul2(r2, __float2half2_rn(-1152.f));
            const uint4 v = *reinterpret_cast<const uint4*>(src + chunk_at<D>(row, ch));
            const uint32_t wd[4] = {bias_codes<FMT>(v.x), bias_codes<FMT>(v.y), bias_codes<FMT>(v.z), bias_codes<FMT>(v.w)};
            uint32_t o[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              o[2 * k] = scaled_pair<FMT, false>(wd[k], r2, o2);
              o[2 * k + 1] = scaled_pair<FMT, true>(wd[k], r2, o2);
            }
            uint8_t* rowp = dst + (ch >> 2) * (128 * 128) + row * 128;
            const int c0 = (ch & 3) * 2;
            const uint4 lo = make_uint4(o[0], o[1], o[2], o[3]), hi = make_uint4(o[4], o[5], o[6], o[7]);
            // the upper half row writes its second chunk first: no bank conflicts
            const int sw = ch >> 2;
            *reinterpret_cast<uint4*>(rowp + (((c0 + sw) ^ (row & 7)) << 4)) = sw ? hi : lo;
            *reinterpret_cast<uint4*>(rowp + (((c0 + 1 - sw) ^ (row & 7)) << 4)) = sw ? lo : hi;
          }
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&k_full[st]);
          mbar_arrive(&stg_empty[0]);
        }
        // values
        wait(&stg_full[1], i, 66);
        wait(&v_empty[st], (i >> 1) + 1, 67);
        {
          const uint8_t* src = smem + C::kStgOff + C::kStg;
          uint8_t* dst = smem + C::kVOff + st * C::kKv;
          constexpr int kL = D / 4, kIt = D / 32;   // lanes of a row, passes of 16 groups of 8 tokens
          const int l = lane % kL;
          const int pos = (s.tile0 + s.t + j) * kPromptTile;
          const bool edge = pos + kPromptTile > w.q.kv || pos < seen;
#pragma unroll
          for (int it = 0; it < kIt; ++it) {
            const int grp = D == 128 ? it * 4 + cw : it * 8 + cw * 2 + lane / kL;
            const __half2 r2 = ratio(mt[grp >> 1].y, ve), o2 = __hmul2(r2, __float2half2_rn(-1152.f));
            uint32_t wd[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const int row = grp * 8 + k;
              wd[k] = *reinterpret_cast<const uint32_t*>(src + chunk_at<D>(row, l >> 2) + 4 * (l & 3));
              // slots past the sequence's tokens may hold anything: as 0 they add 0 * 0
              if (edge && (pos + row >= w.q.kv || pos + row < seen)) wd[k] = 0;
              wd[k] = bias_codes<FMT>(wd[k]);
            }
            uint32_t o[4][4];   // [element][pair of tokens]
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t e01 = __byte_perm(wd[2 * k], wd[2 * k + 1], 0x5140);
              const uint32_t e23 = __byte_perm(wd[2 * k], wd[2 * k + 1], 0x7362);
              o[0][k] = scaled_pair<FMT, false>(e01, r2, o2), o[1][k] = scaled_pair<FMT, true>(e01, r2, o2);
              o[2][k] = scaled_pair<FMT, false>(e23, r2, o2), o[3][k] = scaled_pair<FMT, true>(e23, r2, o2);
            }
            uint8_t* base = dst + (grp >> 3) * (D * 128);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int n = e * (D / 4) + l;
              *reinterpret_cast<uint4*>(base + n * 128 + (((grp & 7) ^ (n & 7)) << 4)) =
                  make_uint4(o[e][0], o[e][1], o[e][2], o[e][3]);
            }
          }
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&v_full[st]);
          mbar_arrive(&stg_empty[1]);
        }
      }
    }
  } else if (warp < kProd) {
    // ---------------- the MMAs of row tile t, from one lane
    const int t = warp - kIssue0;
    if (lane == 0) {
      const uint32_t ts = tmem + 128 * t, to = tmem + 256 + D * t;
      const uint32_t ids = idesc_f16(128), ido = idesc_f16(D);
      const uint32_t qa = smem_u32(smem + t * C::kQ);
      int i = 0;
      uint32_t jt = 0, segs = 0;
      while (walk.next(p, s)) {
        const int live = live_units(walk.w, s, t), units = max(live, live_units(walk.w, s, 1 - t));
        if (live > 0) wait(&q_full[t], segs++, 68);
        for (int j = 0; j < units; ++j, ++i) {
          const int st = i & 1;
          wait(&k_full[st], i >> 1, 69);
          if (j < live) {
            if (jt > 0) wait(&o_done[t], jt - 1, 70);   // P, which lies over S, has been read
            if (ok) {
              tc_fence_after();
              const uint32_t kb = smem_u32(smem + C::kKOff + st * C::kKv);
#pragma unroll
              for (int k = 0; k < D / 16; ++k)
                umma_f16_ss(ts, sw128_desc(qa + (k >> 2) * (128 * 128) + (k & 3) * 32),
                            sw128_desc(kb + (k >> 2) * (128 * 128) + (k & 3) * 32), ids, k != 0);
              umma_commit(&k_empty[st]);
              umma_commit(&s_full[t]);
            }
          } else {
            mbar_arrive(&k_empty[st]);
          }
          wait(&v_full[st], i >> 1, 71);
          if (j < live) {
            wait(&p_full[t], jt, 72);
            if (ok) {
              tc_fence_after();
              const uint32_t vb = smem_u32(smem + C::kVOff + st * C::kKv);
#pragma unroll
              for (int k = 0; k < 8; ++k)
                umma_f16_ts(to, ts + 8 * k, sw128_desc(vb + (k >> 2) * (D * 128) + (k & 3) * 32), ido, j != 0 || k != 0);
              umma_commit(&v_empty[st]);
              umma_commit(&o_done[t]);   // (last: the CTA may end once it has come)
            }
            ++jt;
          } else {
            mbar_arrive(&v_empty[st]);
          }
        }
      }
    }
    __syncwarp();
  } else if (warp == kProd) {
    // ---------------- pages: lane i has page i of a batch of 32
    const int ppt = kPromptTile / p.block, tiles = 32 / ppt, pbytes = p.block * D;
    int i = 0;
    while (walk.next(p, s)) {
      const PromptWork& w = walk.w;
      const int units = max(live_units(w, s, 0), live_units(w, s, 1));
      const PageRun run = read_pages(w.q, p.block, p.window);
      const int pg0 = (s.tile0 + s.t) * ppt;
      auto page_at = [&](int k) {   // page k of the segment, -1 for none
        const int pg = pg0 + k;
        if (k >= units * ppt || pg < run.first || pg >= run.first + run.n) return -1;
        const int id = page_block(p.seqs, s.b, pg, p.num_blocks);
        if (id < 0) set_status(p.status, FL_ERR_DEVICE_CHECK, 55);
        return id;
      };
      auto scales_of = [&](int id) {
        if (id < 0) return make_float2(1.f, 1.f);
        const int64_t at = static_cast<int64_t>(id) * p.heads + s.h;
        return make_float2(p.ks[at], p.vs[at]);
      };
      int id0 = -1, id1 = page_at(lane), id2 = page_at(32 + lane);
      float2 sc0 = make_float2(1.f, 1.f), sc1 = scales_of(id1);
      for (int j = 0; j < units; ++j, ++i) {
        const int k = j % tiles;
        if (k == 0) {
          id0 = id1, id1 = id2;
          sc0 = sc1, sc1 = scales_of(id1);
          id2 = page_at((j / tiles + 2) * 32 + lane);
        }
        const bool mine = lane >= k * ppt && lane < (k + 1) * ppt && id0 >= 0;
        const uint32_t valid = __ballot_sync(0xffffffffu, mine);
        const int row = mine ? static_cast<int>((static_cast<int64_t>(id0) * p.heads + s.h) * p.block) : 0;
        const int from = k * ppt + (lane & 7) * 16 / p.block;
        const float a = __shfl_sync(0xffffffffu, sc0.x, from), v = __shfl_sync(0xffffffffu, sc0.y, from);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (i > 0) wait(&stg_empty[h], i - 1, 73);
          ok = __all_sync(0xffffffffu, ok);
          if (ok) {
            if (lane == 0 && valid) mbar_expect_tx(&stg_full[h], static_cast<uint32_t>(pbytes) * __popc(valid));
            if (h == 0 && lane < 8) meta[(i & 3) * 8 + lane] = make_float2(a, v);
            __syncwarp();
            if (mine)
              tma_load_2d(smem + C::kStgOff + h * C::kStg + (lane - k * ppt) * pbytes, h ? &vmap : &kmap, 0, row, &stg_full[h]);
            __syncwarp();
            if (lane == 0) mbar_arrive(&stg_full[h]);
          }
        }
      }
    }
    // (in the normal course the converters have waited for every copy)
    if (!ok && i > 0)
      for (int h = 0; h < 2; ++h) mbar_wait(&stg_full[h], static_cast<uint32_t>(i - 1) & 1u);
  }

  tc_fence_before();
  cta_sync();
  tc_fence_after();
  if (warp == kIssue0) tmem_dealloc(tmem, 512);
}

template <int FMT, int D>
int launch(const CUtensorMap& km, const CUtensorMap& vm, const AttnParams& p, cudaStream_t s) {
  using C = PrCfg<D>;
  static bool attr_done[64] = {false};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return FL_ERR_CUDA;
  if (dev >= 64 || !attr_done[dev]) {
    if (cudaFuncSetAttribute(k_kv8_prompt<FMT, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem) != cudaSuccess)
      return FL_ERR_CUDA;
    if (dev < 64) attr_done[dev] = true;
  }
  k_kv8_prompt<FMT, D><<<flh::sm_count(), kPrThreads, C::kSmem, s>>>(km, vm, p);
  return cudaGetLastError() == cudaSuccess ? FL_OK : FL_ERR_CUDA;
}

}  // namespace

namespace flkv {

size_t prompt_slot_floats(int head_dim) { return static_cast<size_t>(kPromptRows) * (head_dim + 2); }

int launch_prompt(const CUtensorMap& km, const CUtensorMap& vm, const AttnParams& p, int format, int head_dim, cudaStream_t s) {
  if (format == FL_KV8_E4M3)
    return head_dim == 64 ? launch<FL_KV8_E4M3, 64>(km, vm, p, s) : launch<FL_KV8_E4M3, 128>(km, vm, p, s);
  return head_dim == 64 ? launch<FL_KV8_INT8, 64>(km, vm, p, s) : launch<FL_KV8_INT8, 128>(km, vm, p, s);
}

}  // namespace flkv

// Test hook: the units of a sequence of rows / group tokens, kv of them cached.
extern "C" int fl_kv8_test_units(int n, int kv, int group, int heads, int window, long long u, long long* out) {
  if (!out || n < 0 || kv < 0 || group < 1 || heads < 1 || window < 0) return FL_ERR_ARG;
  const PromptWork w = prompt_work(SeqInfo{0, n, kv}, group, heads, window, 0, 0x7fffffff);
  out[0] = w.items, out[1] = w.per_head;
  if (u < 0 || u >= w.per_head) return FL_OK;
  const int item = w.item_of(u);
  out[2] = item, out[3] = u - w.before(item), out[4] = w.tiles(item), out[5] = w.first_tile(item);
  out[6] = w.lim(item * kPromptRows, kPromptRows), out[7] = w.low(item * kPromptRows);
  return FL_OK;
}
