// Attention over the 8-bit paged cache for many query rows (prompts, chunks):
// the contraction-bound form, on tcgen05.
//
// An item is 256 rows of a kv head (rows are (token, query head of the group),
// so that a group shares its keys) in two tiles of 128, a unit one item x 128
// tokens.  The units of the batch lie in one line and each of the persistent
// CTAs (one an SM) takes an equal run of them, so ragged batches, the causal
// triangle and few rows over a long context all fill the GPU; an item that
// several CTAs share leaves partials, which a second, small kernel joins in CTA
// order (one CTA would take 20 us to add up 19 partials of 131 KB).
//
// Per unit: S = Q K^T (128 x 128 a row tile, fp32 in tensor memory), softmax
// with the running maximum and sum, P as f16 back into S's columns, O += P V
// (P from tensor memory, O there too).  Codes become f16 once per CTA and unit,
// in shared memory, and serve both row tiles.  Warps:
//   0..3, 4..7  softmax of row tile 0, 1: a thread has a row.  The reference
//               that weights are taken against moves only when a maximum has
//               passed it by 2^8, so one pass over S does: the maximum of 64
//               columns, their weights, P back; where a reference has moved, P,
//               O and the sum are rescaled by the power of two
//   8..11       convert key rows as they are (K-major)
//   12..15      convert values, transposed
//               (tokens along K) with byte permutes: the order of output
//               columns is free, so value element 4 l + j goes to row j D/4 + l,
//               which makes the writes conflict-free
//   16, 17      issue the MMAs of row tile 0, 1
//   18          copies pages by TMA into a staging tile for keys and for values
//   19          walks the CTA's units and publishes their segments to the others
//
// Scales: with e_b the power of two in a block's scale and e_ref the largest of
// the segment's, codes are multiplied by 2^(e_b - e_ref + k) as they
// become f16 (exact down to 2^-24 of f16: blocks whose scales are 2^20 apart)
// and the reference goes into the row's factor or the output.  Mantissas of
// scales other than powers of two go into S, for the sequences that have them.
// q as in the kernel for few rows.  P is f16 (2^-11, the output's rounding is
// 2^-8) times 2^6, and up to 2^15; its fp32 sum is taken before.
//
// Measured (heads of 128, e4m3): 2048 tokens after 14336, 32 query and 8 kv
// heads, 394 us, 1.31 PFLOP/s; a prompt of 4095 tokens, 32 kv heads, 181 us, 0.76
// PFLOP/s; 8192 tokens 618 us, 0.89 (in a chain of calls).  A unit takes 3.3K cycles where its MMAs take
// 2.0K: the softmax warps' latency (two a scheduler; more do not fit the
// registers) is what bounds it.  A segment costs 15K cycles beside its units (q
// in, the masked units, the output), 4 to 7 of them a CTA in the prompts, and a
// call 8 us before its first unit.
#include "fl_kv8_prompt.cuh"
#include "fl_tc.cuh"

using namespace flkv;

namespace {

constexpr int kPrThreads = 640;
constexpr int kConv0 = 8, kIssue0 = 16, kProd = 18, kPlan = 19;   // first warps of the roles
constexpr int kConvWarps = 4;                         // for keys, and for values
// Registers a thread: all at launch (the build fails where the compiler takes
// another count), then by role (warps 16..19 share one count)
constexpr int kRegs = 96, kRegsSoftmax = 136, kRegsConv = 64, kRegsRest = 80;
static_assert(256 * kRegsSoftmax + 64 * kConvWarps * kRegsConv + 128 * kRegsRest <= kPrThreads * kRegs, "register pool");
constexpr int kPromptLeast = 2;                       // fewest units of a CTA
constexpr float kBias = 6.f;                          // P is at most 2^kBias when its reference is taken
constexpr float kSlack = 8.f;                         // and 2^(kBias + kSlack) before it is taken anew

template <int D>
struct PrCfg {
  static constexpr int kQ = 128 * D * 2;       // a row tile of q
  static constexpr int kKv = 128 * D * 2;      // keys or values of a unit as f16
  static constexpr int kStg = 128 * D;         // their codes
  static constexpr int kKOff = 2 * kQ;         // two stages
  static constexpr int kVOff = kKOff + 2 * kKv;
  static constexpr int kStgOff = kVOff + 2 * kKv;
  static constexpr int kMetaOff = kStgOff + 2 * kStg;      // [8 units][8 slices of 16 tokens]: mantissas of scales
  static constexpr int kRatioOff = kMetaOff + 8 * 8 * 16;   // [8][8]: the codes' multipliers, f16 pairs
  static constexpr int kSegOff = kRatioOff + 8 * 8 * 8;    // [4] segments
  static constexpr int kBarOff = kSegOff + 4 * 64;
  static constexpr int kBars = 4 + 8 + 2 + 4 + 4 + 4 + 8;
  static constexpr int kSmem = kBarOff + kBars * 8 + 16;
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
__device__ __forceinline__ void tmem_ld32_issue(uint32_t taddr, float (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
        "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15]), "=f"(r[16]),
        "=f"(r[17]), "=f"(r[18]), "=f"(r[19]), "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]), "=f"(r[24]),
        "=f"(r[25]), "=f"(r[26]), "=f"(r[27]), "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld32_wait(float (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(r[0]), "+f"(r[1]), "+f"(r[2]), "+f"(r[3]), "+f"(r[4]), "+f"(r[5]), "+f"(r[6]), "+f"(r[7]),
                 "+f"(r[8]), "+f"(r[9]), "+f"(r[10]), "+f"(r[11]), "+f"(r[12]), "+f"(r[13]), "+f"(r[14]), "+f"(r[15]),
                 "+f"(r[16]), "+f"(r[17]), "+f"(r[18]), "+f"(r[19]), "+f"(r[20]), "+f"(r[21]), "+f"(r[22]), "+f"(r[23]),
                 "+f"(r[24]), "+f"(r[25]), "+f"(r[26]), "+f"(r[27]), "+f"(r[28]), "+f"(r[29]), "+f"(r[30]), "+f"(r[31])
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
// 64 columns, and the wait for them, in one: the registers need no tie to a wait
// of its own (which cost a move for each).
__device__ __forceinline__ void tmem_ld64(uint32_t taddr, float (&a)[32], float (&b)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%64];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%65];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(a[0]), "=f"(a[1]), "=f"(a[2]), "=f"(a[3]), "=f"(a[4]), "=f"(a[5]), "=f"(a[6]), "=f"(a[7]), "=f"(a[8]), "=f"(a[9]), "=f"(a[10]), "=f"(a[11]), "=f"(a[12]), "=f"(a[13]), "=f"(a[14]), "=f"(a[15]), "=f"(a[16]), "=f"(a[17]), "=f"(a[18]), "=f"(a[19]), "=f"(a[20]), "=f"(a[21]), "=f"(a[22]), "=f"(a[23]), "=f"(a[24]), "=f"(a[25]), "=f"(a[26]), "=f"(a[27]), "=f"(a[28]), "=f"(a[29]), "=f"(a[30]), "=f"(a[31]),
        "=f"(b[0]), "=f"(b[1]), "=f"(b[2]), "=f"(b[3]), "=f"(b[4]), "=f"(b[5]), "=f"(b[6]), "=f"(b[7]), "=f"(b[8]), "=f"(b[9]), "=f"(b[10]), "=f"(b[11]), "=f"(b[12]), "=f"(b[13]), "=f"(b[14]), "=f"(b[15]), "=f"(b[16]), "=f"(b[17]), "=f"(b[18]), "=f"(b[19]), "=f"(b[20]), "=f"(b[21]), "=f"(b[22]), "=f"(b[23]), "=f"(b[24]), "=f"(b[25]), "=f"(b[26]), "=f"(b[27]), "=f"(b[28]), "=f"(b[29]), "=f"(b[30]), "=f"(b[31])
      : "r"(taddr), "r"(taddr + 32)
      : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

template <int N>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// A run of units of one item inside the CTA's units, as the roles need it.
struct __align__(16) Segment {
  int units;       // with work (row tile 0 or 1); -1: no more segments
  int live[2];     // of them, those in which row tile 0, 1 has a visible token
  int tile;        // tile of the first unit
  int b, h;        // sequence, kv head
  int row0, rows;  // first row of the item; rows of the sequence
  int start;       // first query row (token) of the sequence
  int past, kv;    // position of that row; tokens of the sequence
  int slot;        // the partial to write, or -1: the item is whole, write its output
  int ke, ve;      // largest powers of two of its units' key and value scales
  int general;     // the scales have mantissas
  int meta;        // place of the first unit's scales
};
static_assert(sizeof(Segment) == 64, "segment ring");

// What the joining kernel needs of the item that CTA c begins and others go on
// with: CTA c writes entry c, with last = -1 if there is none.
struct __align__(16) JoinItem {
  int last;                  // the last CTA of the item
  int start, rows, row0, h;  // as in the segment
  int pad[3];
};

struct PromptWalk {
  long long u, end, base;
  int b;
  PromptWork w;
  // the item that unit u lies in: of head h, `nt` units from the head's `at` on
  int h, item, nt;
  long long at;
  __device__ void load(const AttnParams& p) {
    w = prompt_work(seq_info(p.seqs, b, p.block), p.group, p.heads, p.window, p.rows_lo, p.rows_hi);
  }
  // Finds unit u's item; u lies in sequence b, which is loaded.  A warp's 32
  // lanes look at 32 items at a time.
  __device__ void find() {
    const long long local = u - base;
    h = local < (1ll << 31) && w.per_head < (1ll << 31)
            ? static_cast<int>(static_cast<unsigned>(local) / static_cast<unsigned>(w.per_head))
            : static_cast<int>(local / w.per_head);
    const long long in_head = local - h * w.per_head;
    int lo = 0, n = w.items;   // the item is one of [lo, lo + n)
    while (n > 1) {
      const int step = (n + 31) / 32, at_lane = lo + min(static_cast<int>(threadIdx.x & 31) * step, n);
      const uint32_t begun = __ballot_sync(0xffffffffu, at_lane < lo + n && w.before(at_lane) <= in_head);
      const int k = 31 - __clz(begun);   // (lane 0's always has)
      n = min(step, n - k * step);
      lo += k * step;
    }
    item = lo;
    at = w.before(item);
    nt = static_cast<int>(w.before(item + 1) - at);
  }
  // Moves to the next item; false past the last.
  __device__ bool step(const AttnParams& p) {
    at += nt;
    if (++item == w.items) {
      item = 0, at = 0;
      if (++h == p.heads) {
        h = 0;
        base += w.per_head * p.heads;
        do {
          if (++b >= p.seqs.B) return false;
          load(p);
        } while (w.items == 0);
      }
    }
    nt = static_cast<int>(w.before(item + 1) - at);
    return true;
  }
  __device__ bool next(const AttnParams& p, Segment& s, long long ubeg) {
    s.units = -1;
    if (u >= end) return false;
    const int t = static_cast<int>(u - base - h * w.per_head - at);
    const int n = static_cast<int>(min(static_cast<long long>(nt - t), end - u));
    s.b = b;
    s.h = h;
    s.row0 = item * kPromptRows;
    s.rows = w.rows;
    s.tile = w.first_tile(item) + t;
    for (int k = 0; k < 2; ++k) {
      const int r0 = s.row0 + 128 * k;
      s.live[k] = r0 >= w.rows ? 0 : min(max((max(w.lim(r0, 128), 0) + kPromptTile - 1) / kPromptTile - s.tile, 0), n);
    }
    s.units = max(s.live[0], s.live[1]);
    s.start = w.q.start, s.past = w.past, s.kv = w.q.kv;
    // a CTA's partials: 0 for an item begun by the CTAs before, 1 for one begun here
    s.slot = n == nt ? -1 : 2 * static_cast<int>(blockIdx.x) + (u - t < ubeg ? 0 : 1);
    u += n;
    if (u < end && t + n == nt) step(p);
    return true;
  }
};

// (behind the partials)
template <int D>
__device__ __forceinline__ JoinItem* join_items(const AttnParams& p, int ctas) {
  return reinterpret_cast<JoinItem*>(p.part + 2 * static_cast<size_t>(ctas) * PrCfg<D>::kSlot);
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
  // No static shared memory: the dynamic part begins the CTA's window, on the
  // 1024-byte boundary that the swizzled tiles need (checked below).
  extern __shared__ __align__(1024) uint8_t smem[];
  float4* meta = reinterpret_cast<float4*>(smem + C::kMetaOff);   // the key's, log2 of the value's, one over the value's
  uint2* ratios = reinterpret_cast<uint2*>(smem + C::kRatioOff);
  Segment* segs = reinterpret_cast<Segment*>(smem + C::kSegOff);
  uint64_t* stg_full = reinterpret_cast<uint64_t*>(smem + C::kBarOff);   // [keys, values]
  uint64_t* stg_empty = stg_full + 2;
  uint64_t* k_full = stg_empty + 2;      // [stage]
  uint64_t* k_empty = k_full + 2;
  uint64_t* v_full = k_empty + 2;
  uint64_t* v_empty = v_full + 2;
  uint64_t* q_full = v_empty + 2;        // [row tile]
  // [row tile][buffer]: with one barrier a tile a phase could complete twice before its waiter looks
  uint64_t* s_full = q_full + 2;
  uint64_t* p_full = s_full + 4;
  uint64_t* o_done = p_full + 4;
  uint64_t* seg_full = o_done + 4;       // [4]
  uint64_t* seg_empty = seg_full + 4;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(seg_empty + 4);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_launch_dependents();
  if (warp == kProd && lane == 0) prefetch_map(&kmap), prefetch_map(&vmap);
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&stg_full[i], 1);
      mbar_init(&stg_empty[i], kConvWarps);
      mbar_init(&k_full[i], kConvWarps);
      mbar_init(&k_empty[i], 2);
      mbar_init(&v_full[i], kConvWarps);
      mbar_init(&v_empty[i], 2);
      mbar_init(&q_full[i], 4);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
      mbar_init(&o_done[i], 1);
      mbar_init(&seg_full[i], 1);
      mbar_init(&seg_empty[i], kPlan);   // one arrival of every warp before the planner
    }
    fence_mbar_init();
  }
  pdl_wait();
  if (smem_u32(smem) & 1023u) {
    if (tid == 0) {
      set_status(p.status, FL_ERR_DEVICE_CHECK, 56);
      join_items<D>(p, gridDim.x)[blockIdx.x].last = -1;
    }
    return;
  }
  if (warp == kPlan && lane == 0) join_items<D>(p, gridDim.x)[blockIdx.x].last = -1;   // until the plan says more
  const Start start = find_start<kPrThreads>(reinterpret_cast<long long*>(smem + C::kStgOff), p.seqs.B, blockIdx.x, gridDim.x, kPromptLeast, [&](int b) {
    const SeqInfo q = seq_info(p.seqs, b, p.block);
    if (q.bad && blockIdx.x == 0) set_status(p.status, FL_ERR_DEVICE_CHECK, 58);
    return prompt_work(q, p.group, p.heads, p.window, p.rows_lo, p.rows_hi).per_head * p.heads;
  });
  if (static_cast<int>(blockIdx.x) >= start.P) return;
  fence_proxy_async();   // the scan's numbers lay where pages are copied to
  if (warp == kIssue0) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  cta_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;   // S of row tile t and half b at 128 t + 64 b, P over it, O at 256 + D t
  bool ok = true;   // false after a wait ran out: nothing is waited for or issued any more
  auto wait_one = [&](uint64_t* bar, uint32_t phase, int where) {
    if (ok && !mbar_wait_many(bar, phase & 1u)) {
      set_status(p.status, FL_ERR_TIMEOUT, where);
      ok = false;
    }
  };
  auto wait = [&](uint64_t* bar, uint32_t phase, int where) {   // of a whole warp: its lanes go on or give up together
    wait_one(bar, phase, where);
    ok = __all_sync(0xffffffffu, ok);
  };

  if (warp < kConv0) {
    // ---------------- softmax and output: a thread has row r of row tile t
    regs_up<kRegsSoftmax>();
    const int t = warp >> 2, r = (warp & 3) * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t to = tmem + lanes + 256 + D * t;
    uint32_t js = 0;    // half units of this row tile so far
    for (int seg = 0; ok; ++seg) {
      wait(&seg_full[seg & 3], seg >> 2, 59);
      const Segment& s = segs[seg & 3];
      if (!ok || s.units < 0) break;
      const int live = s.live[t];
      const bool general = s.general != 0;
      float a = 0.f, far = 1.f;   // what S is times to be a score, as far * a with a <= 1
      if (live > 0) {
        // The warp's 32 rows of q: copied to their places in the tile, kL lanes a
        // row, then there times a power of two a row and the sign of the scale, as
        // f16.  In short loops: code that runs once a segment is fetched at some 7
        // cycles an instruction.
        constexpr int kL = D / 8, kR = 32 / kL, kN = 32 / kR;
        const int own = s.row0 + 128 * t + r, tok = own / p.group;
        const unsigned long long from =
            own < s.rows ? reinterpret_cast<unsigned long long>(p.q + (static_cast<int64_t>(s.start) + tok) * p.qs +
                                                                static_cast<int64_t>(s.h * p.group + own - tok * p.group) * D)
                         : 0ull;
        uint8_t* tile = smem + t * C::kQ;
        auto place = [&](int rr, int ch) {   // 16 bytes of a row of the tile
          return reinterpret_cast<uint4*>(tile + rr * 128 + (ch >> 3) * (128 * 128) + (((ch & 7) ^ (rr & 7)) << 4));
        };
#pragma unroll 1
        for (int i = 0; i < kN; ++i) {
          const unsigned long long row = __shfl_sync(0xffffffffu, from, kR * i + lane / kL);
          cp_async16(place((warp & 3) * 32 + kR * i + lane / kL, lane % kL),
                     reinterpret_cast<const uint4*>(row ? row : reinterpret_cast<unsigned long long>(p.q)) + lane % kL, row != 0);
        }
        cp_async_wait_all();
        __syncwarp();
        // from here a lane has its own row (in place, without bank conflicts)
        uint32_t mine = 0;   // the largest magnitude's bits
#pragma unroll 4
        for (int i = 0; i < kL; ++i) {
          const uint4 x = *place(r, i);
          mine = __vmaxu2(mine, __vmaxu2(__vmaxu2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu), __vmaxu2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu)));
        }
        mine = max(mine & 0xffffu, mine >> 16);
        const float down = copysignf(pow2i(-row_exponent(mine)), p.scale2);
#pragma unroll 4
        for (int i = 0; i < kL; ++i) {
          const uint4 x = *place(r, i);
          auto pair = [&](uint32_t v) {
            return pack_f16(__uint_as_float(v << 16) * down, __uint_as_float(v & 0xffff0000u) * down);
          };
          *place(r, i) = make_uint4(pair(x.x), pair(x.y), pair(x.z), pair(x.w));
        }
        a = fabsf(p.scale2) * pow2i(row_exponent(mine)) * pow2i(max(s.ke - code_shift<FMT>(), -126));
        a = fmaxf(a, 1.1754943508222875e-38f);   // (not 0: -inf of a masked column stays -inf)
        far = fmaxf(a, 1.f), a = fminf(a, 1.f);
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_full[t]);
      }
      // half units [plain_begin, plain_end) of which every row of the tile sees every token
      int plain_begin = 0, plain_end;
      {
        const int r0 = s.row0 + 128 * t, pos = s.tile * kPromptTile;
        plain_end = (s.past + r0 / p.group + 1 - pos) >> 6;
        if (p.window) plain_begin = (s.past + min(r0 + 127, s.rows - 1) / p.group + 1 - p.window - pos + 63) >> 6;
      }
      // S is below 2^24 (2^25 with mantissas).  With a factor of at most 1 a score is
      // too, and the rounding of its reference, an integer, leaves P within f16.
      // Scores beyond have lost their fractions in fp32; for them S takes what the
      // factor has above 1 first, so that all are rounded alike (in one rounding with
      // the subtraction of the reference, weights of equal scores of 2^26 came out
      // infinite or 0).
      const bool any_far = __any_sync(0xffffffffu, far > 1.f);
      float m = -INFINITY, l = 0.f;   // weights are 2^(x - m); the reference m is an integer, about kBias below a maximum
      for (int j = 0; j < 2 * live; ++j, ++js) {
        const uint32_t ts = tmem + lanes + 128 * t + 64 * (js & 1);
        wait(&s_full[2 * t + (js & 1)], js >> 1, 61);
        tc_fence_after();
        // The loops of all roles are kept short on purpose: unrolled, they do not
        // fit the instruction cache together, and a unit took twice as long.  And
        // they spill no register: little of the L1 is left beside the tiles, so
        // that a spilled value comes back from L2.
        // Mantissas of scales: the keys' multiply S, the values' add their log2 to
        // the exponent of the weight and leave its sum below.  This is done in
        // tensor memory, so that no register of the loop is touched: as a branch on
        // the values themselves it cost a sixth (4095-token prompt 220 us, not 184).
        const float4* mt = meta + ((s.meta + (j >> 1)) & 7) * 8 + 4 * (j & 1);   // of 16 tokens each
        if (general || any_far) {
          const float down = rcp_approx(a);
#pragma unroll 1
          for (int k = 0; k < 8; ++k) {
            const float mul = general ? mt[k >> 1].x * far : far, add = general ? mt[k >> 1].y * down : 0.f;
            uint32_t o[8];
            tmem_ld8_issue(ts + 8 * k, o);
            tmem_ld8_wait(o);
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = __float_as_uint(fmaf(__uint_as_float(o[i]), mul, add));
            tmem_st8(ts + 8 * k, o);
          }
          tmem_wait_st();
        }
        float x[2][32];
        tmem_ld64(ts, x[0], x[1]);
        if (j >= plain_end || j < plain_begin) {
          // -inf where this row does not see the token: columns [lo, hi) are seen
          const int pos = s.tile * kPromptTile + 64 * j;
          const int hi = s.past + min(s.row0 + 128 * t + r, s.rows - 1) / p.group + 1 - pos;
          const int lo = p.window ? hi - p.window : -0x40000000;
#pragma unroll
          for (int i = 0; i < 64; ++i)
            if (i >= hi || i < lo) x[i >> 5][i & 31] = -INFINITY;
        }
        float mx4[4] = {x[0][0], x[0][1], x[1][0], x[1][1]};
#pragma unroll
        for (int i = 1; i < 16; ++i) {
          mx4[i & 1] = max3(mx4[i & 1], x[0][2 * i], x[0][2 * i + 1]);
          mx4[2 + (i & 1)] = max3(mx4[2 + (i & 1)], x[1][2 * i], x[1][2 * i + 1]);
        }
        const float top = max3(fmaxf(mx4[0], mx4[1]), mx4[2], mx4[3]) * a;
        if (__any_sync(0xffffffffu, top - m > kBias + kSlack)) {
          // a maximum has outgrown its reference: the rows of O and the sum move
          const float nm = top - m > kBias + kSlack ? ceilf(top - kBias) : m;
          const float f = nm == m ? 1.f : exp2_approx(m - nm);
          m = nm;
          l *= f;
          if (j > 0) {
            wait(&o_done[2 * t + ((js - 1) & 1)], (js - 1) >> 1, 62);
            tc_fence_after();
#pragma unroll 1
            for (int k = 0; k < D / 8; ++k) {
              uint32_t o[8];
              tmem_ld8_issue(to + 8 * k, o);
              tmem_ld8_wait(o);
#pragma unroll
              for (int i = 0; i < 8; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
              tmem_st8(to + 8 * k, o);
            }
          }
        }
        const float mm = m == -INFINITY ? 0.f : -m;
        float2 lsum[4];   // of 16 tokens each
#pragma unroll
        for (int k = 0; k < 2; ++k) {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float2 e = __ffma2_rn(make_float2(x[k][2 * i], x[k][2 * i + 1]), make_float2(a, a), make_float2(mm, mm));
            x[k][2 * i] = exp2_approx(e.x), x[k][2 * i + 1] = exp2_approx(e.y);
            const float2 w = make_float2(x[k][2 * i], x[k][2 * i + 1]);
            lsum[2 * k + (i >> 3)] = (i & 7) == 0 ? w : __fadd2_rn(lsum[2 * k + (i >> 3)], w);
          }
          uint32_t pk[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) pk[i] = pack_f16(x[k][2 * i], x[k][2 * i + 1]);
          tmem_st16(ts + 16 * k, pk);   // over columns of S that have been read
        }
        float part[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) part[k] = lsum[k].x + lsum[k].y;
        if (general)
#pragma unroll
          for (int k = 0; k < 4; ++k) part[k] *= mt[k].z;
        l += (part[0] + part[1]) + (part[2] + part[3]);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[2 * t + (js & 1)]);
      }

      // ---------------- the rows' output, or their partial
      if (live > 0) {
        wait(&o_done[2 * t], (js - 2) >> 1, 63);       // (js is even: the last use of either buffer)
        wait(&o_done[2 * t + 1], (js - 2) >> 1, 63);
        tc_fence_after();
      }
      const float back = pow2i(max(s.ve - code_shift<FMT>(), -126));
      if (s.slot < 0) {
        // The warp's rows as bf16 over its rows of q, which is not needed any more,
        // then out, kL lanes a row.
        const int row = s.row0 + 128 * t + r, tok = min(row, s.rows - 1) / p.group;
        const float inv = l == 0.f ? 0.f : back / l;   // 0: no token (a NaN is not)
        const int64_t tk = static_cast<int64_t>(s.start) + tok;
        const int hd = s.h * p.group + row - tok * p.group;
        const unsigned long long into =
            row < s.rows ? reinterpret_cast<unsigned long long>(p.out + tk * p.os + static_cast<int64_t>(hd) * D) : 0ull;
        if (row < s.rows && p.lse) p.lse[tk * p.Hq + hd] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
        uint8_t* tile = smem + t * C::kQ;
#pragma unroll 1
        for (int i = 0; i < D / 32; ++i) {
          // elements 32 i .. 32 i + 31: columns 8 i .. 8 i + 7 of each quarter
          uint32_t o[4][8];
#pragma unroll
          for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int k = 0; k < 8; ++k) o[q][k] = 0;
          if (live > 0) {
#pragma unroll
            for (int q = 0; q < 4; ++q) tmem_ld8_issue(to + q * (D / 4) + 8 * i, o[q]);
#pragma unroll
            for (int q = 0; q < 4; ++q) tmem_ld8_wait(o[q]);
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t v[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const __nv_bfloat162 z = __floats2bfloat162_rn(__uint_as_float(o[2 * (q & 1)][2 * k + (q >> 1)]) * inv,
                                                             __uint_as_float(o[2 * (q & 1) + 1][2 * k + (q >> 1)]) * inv);
              v[q] = *reinterpret_cast<const uint32_t*>(&z);
            }
            const int ch = 4 * i + k;
            *reinterpret_cast<uint4*>(tile + r * 128 + (ch >> 3) * (128 * 128) + (((ch & 7) ^ (r & 7)) << 4)) =
                make_uint4(v[0], v[1], v[2], v[3]);
          }
        }
        __syncwarp();
        constexpr int kL = D / 8, kR = 32 / kL, kN = 32 / kR;
#pragma unroll 1
        for (int i = 0; i < kN; ++i) {
          const unsigned long long dst = __shfl_sync(0xffffffffu, into, kR * i + lane / kL);
          const int rr = (warp & 3) * 32 + kR * i + lane / kL, ch = lane % kL;
          if (dst)
            reinterpret_cast<uint4*>(dst)[ch] = *reinterpret_cast<const uint4*>(
                tile + rr * 128 + (ch >> 3) * (128 * 128) + (((ch & 7) ^ (rr & 7)) << 4));
        }
        __syncwarp();
      } else {
        float* slot = p.part + static_cast<size_t>(s.slot) * C::kSlot + 128 * t + r;
#pragma unroll 1
        for (int i = 0; i < D / 32; ++i) {
          float o[32];
          if (live > 0) {
            tmem_ld32_issue(to + 32 * i, o);
            tmem_ld32_wait(o);
          }
#pragma unroll
          for (int k = 0; k < 32; ++k) __stcg(slot + (32 * i + k) * kPromptRows, live > 0 ? o[k] * back : 0.f);
        }
        __stcg(slot + D * kPromptRows, m);
        __stcg(slot + (D + 1) * kPromptRows, l);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&seg_empty[seg & 3]);
    }
  } else if (warp < kIssue0) {
    // ---------------- convert
    regs_down<kRegsConv>();
    const bool values = warp >= kConv0 + kConvWarps;
    const int cw = (warp - kConv0) % kConvWarps;
    int i = 0;
    for (int seg = 0; ok; ++seg) {
      wait(&seg_full[seg & 3], seg >> 2, 59);
      const Segment& s = segs[seg & 3];
      if (!ok || s.units < 0) break;
      SeqInfo q;
      q.kv = s.kv, q.n = s.kv - s.past, q.start = 0;
      const int seen = first_seen(q, p.window), units = s.units;
      int pos = s.tile * kPromptTile;
      __syncwarp();
      if (lane == 0) mbar_arrive(&seg_empty[seg & 3]);
      if (!values) {
        for (int j = 0; j < units; ++j, ++i) {
          const int st = i & 1;
          wait(&stg_full[0], i, 64);
          wait(&k_empty[st], (i >> 1) + 1, 65);
          const uint8_t* src = smem + C::kStgOff;
          uint8_t* dst = smem + C::kKOff + st * C::kKv;
          const uint2* rt = ratios + (i & 7) * 8;
          // a warp has two slices of 16 tokens; eight lanes take one 16-byte
          // chunk of eight rows, free of bank conflicts in both layouts
          constexpr int kCh = D / 16;   // chunks of a row
#pragma unroll 2
          for (int it = 0; it < kCh; ++it) {
            const int task = it * 32 + lane, ch = (task >> 3) % kCh, row = cw * 32 + task / (8 * kCh) * 8 + (lane & 7);
            const uint32_t rr = rt[row >> 4].x;
            const __half2 r2 = *reinterpret_cast<const __half2*>(&rr), o2 = __hmul2(r2, __float2half2_rn(-1152.f));
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
            *reinterpret_cast<uint4*>(rowp + ((c0 ^ (row & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
            *reinterpret_cast<uint4*>(rowp + (((c0 + 1) ^ (row & 7)) << 4)) = make_uint4(o[4], o[5], o[6], o[7]);
          }
          fence_proxy_async();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&stg_empty[0]);
            mbar_arrive(&k_full[st]);
          }
        }
      } else {
        for (int j = 0; j < units; ++j, ++i, pos += kPromptTile) {
          const int st = i & 1;
          wait(&stg_full[1], i, 66);
          wait(&v_empty[st], (i >> 1) + 1, 67);
          const uint8_t* src = smem + C::kStgOff + C::kStg;
          uint8_t* dst = smem + C::kVOff + st * C::kKv;
          const uint2* rt = ratios + (i & 7) * 8;
          // lanes of a row; groups of 8 tokens a pass; passes
          constexpr int kL = D / 4, kPer = 32 / kL * kConvWarps, kIt = 16 / kPer;
          const int l = lane % kL;
          const bool edge = pos + kPromptTile > q.kv || pos < seen;
#pragma unroll 1
          for (int it = 0; it < kIt; ++it) {
            const int grp = it * kPer + cw * (32 / kL) + lane / kL;
            const uint32_t rr = rt[grp >> 1].y;
            const __half2 r2 = *reinterpret_cast<const __half2*>(&rr), o2 = __hmul2(r2, __float2half2_rn(-1152.f));
            uint32_t wd[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) wd[k] = *reinterpret_cast<const uint32_t*>(src + chunk_at<D>(grp * 8 + k, l >> 2) + 4 * (l & 3));
            if (edge) {
              // slots past the sequence's tokens may hold anything: as 0 they add 0 * 0
#pragma unroll
              for (int k = 0; k < 8; ++k)
                if (pos + grp * 8 + k >= q.kv || pos + grp * 8 + k < seen) wd[k] = 0;
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) wd[k] = bias_codes<FMT>(wd[k]);
            uint32_t o[4][4];   // [element][pair of tokens]
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t e01 = __byte_perm(wd[2 * k], wd[2 * k + 1], 0x5140);
              const uint32_t e23 = __byte_perm(wd[2 * k], wd[2 * k + 1], 0x7362);
              o[0][k] = scaled_pair<FMT, false>(e01, r2, o2), o[1][k] = scaled_pair<FMT, true>(e01, r2, o2);
              o[2][k] = scaled_pair<FMT, false>(e23, r2, o2), o[3][k] = scaled_pair<FMT, true>(e23, r2, o2);
            }
            uint8_t* base = dst + (grp >> 3) * (D * 128) + l * 128 + (((grp & 7) ^ (l & 7)) << 4);   // (D/4 is a multiple of 8)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              *reinterpret_cast<uint4*>(base + e * (D / 4) * 128) = make_uint4(o[e][0], o[e][1], o[e][2], o[e][3]);
          }
          fence_proxy_async();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&stg_empty[1]);
            mbar_arrive(&v_full[st]);
          }
        }
      }
    }
  } else {
    regs_down<kRegsRest>();
    if (warp < kProd) {
      // ---------------- the MMAs of row tile t, in half units of 64 tokens.  S has
      // two buffers, so that the softmax finds the next half ready: when P of
      // half n has come, O += P V of it, then S of half n + 2 into its place.
      // (The whole warp walks through and an elected lane issues: the
      // descriptors stay in uniform registers.  With one lane in a branch of its
      // own an MMA took 110 cycles to issue, 64 is its time.)
      const int t = __shfl_sync(0xffffffffu, warp - kIssue0, 0);
      const uint32_t ts = tmem + 128 * t, to = tmem + 256 + D * t;
      const uint64_t qd = sw128_desc(smem_u32(smem + t * C::kQ));
      const uint64_t kd0 = sw128_desc(smem_u32(smem + C::kKOff)), vd0 = sw128_desc(smem_u32(smem + C::kVOff));
      int i = 0;                       // first unit of the segment
      uint32_t ju = 0, lived = 0;      // units and segments with work of this row tile so far
      for (int seg = 0; ok; ++seg) {
        wait(&seg_full[seg & 3], seg >> 2, 59);
        const Segment& s = segs[seg & 3];
        const int units = __shfl_sync(0xffffffffu, s.units, 0), live = __shfl_sync(0xffffffffu, s.live[t], 0);
        if (!ok || units < 0) break;
        __syncwarp();
        if (lane == 0) mbar_arrive(&seg_empty[seg & 3]);
        auto scores = [&](int unit, int b) {   // S of half b of a unit
          tc_fence_after();
          if (ok && elect_one()) {
            const uint64_t kd = kd0 + (((unit & 1) * C::kKv + b * (64 * 128)) >> 4);
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
              umma_f16_ss(ts + 64 * b, qd + (((k >> 2) * (128 * 128) + (k & 3) * 32) >> 4),
                          kd + (((k >> 2) * (128 * 128) + (k & 3) * 32) >> 4), idesc_f16(64), k != 0);
            if (b) umma_commit(&k_empty[unit & 1]);
            umma_commit(&s_full[2 * t + b]);
          }
          __syncwarp();
        };
        if (units > 0) wait(&k_full[i & 1], i >> 1, 69);
        if (live > 0) {
          wait(&q_full[t], lived++, 68);
          scores(i, 0);
          scores(i, 1);
        }
#pragma unroll 1
        for (int j = 0; j < units; ++j) {
          const int unit = i + j, st = unit & 1;
          wait(&v_full[st], unit >> 1, 71);
          if (j + 1 < units) wait(&k_full[st ^ 1], (unit + 1) >> 1, 69);
          if (j < live) {
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              wait(&p_full[2 * t + b], ju, 72);
              tc_fence_after();
              if (ok && elect_one()) {
                const uint64_t vd = vd0 + ((st * C::kKv + b * (D * 128)) >> 4);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  umma_f16_ts(to, ts + 64 * b + 8 * k, vd + ((k * 32) >> 4), idesc_f16(D), j != 0 || b != 0 || k != 0);
                if (b) umma_commit(&v_empty[st]);
                umma_commit(&o_done[2 * t + b]);   // (last: the CTA may end once it has come)
              }
              __syncwarp();
              if (j + 1 < live) {
                wait(&o_done[2 * t + b], ju, 70);   // P, which lies over S, has been read
                scores(unit + 1, b);
              }
            }
            ++ju;
          } else if (lane == 0) {
            mbar_arrive(&v_empty[st]);
          }
          // units past this row tile's: their keys are not read either
          if (lane == 0) {
            if (j == 0 && live == 0) mbar_arrive(&k_empty[st]);
            if (j + 1 < units && j + 1 >= live) mbar_arrive(&k_empty[st ^ 1]);
          }
          __syncwarp();
        }
        i += units;
      }
    } else if (warp == kProd) {
      // ---------------- pages: lane i has page i of a batch of 32
      const int ppt = kPromptTile / p.block, tiles = 32 / ppt, pbytes = p.block * D;
      int i = 0;
      for (int seg = 0; ok; ++seg) {
        wait(&seg_full[seg & 3], seg >> 2, 59);
        const Segment& s = segs[seg & 3];
        const int units = s.units, b = s.b, h = s.h, ke = s.ke, ve = s.ve;
        const bool general = s.general != 0;
        if (!ok || units < 0) break;
        SeqInfo q;
        q.kv = s.kv, q.n = s.kv - s.past, q.start = 0;
        const PageRun run = read_pages(q, p.block, p.window);
        const int pg0 = s.tile * ppt;
        __syncwarp();
        if (lane == 0) mbar_arrive(&seg_empty[seg & 3]);
        auto page_at = [&](int k) {   // page k of the segment, -1 for none
          const int pg = pg0 + k;
          if (k >= units * ppt || pg < run.first || pg >= run.first + run.n) return -1;
          const int id = page_block(p.seqs, b, pg, p.num_blocks);
          if (id < 0) set_status(p.status, FL_ERR_DEVICE_CHECK, 55);
          return id;
        };
        // 2^(e - e_ref + shift), 0 below f16 (pages that are not read have a scale of 1, which may exceed e_ref)
        auto ratio = [&](float scale, int e_ref) {
          return __float2half2_rn(pow2i(max(min(scale_exponent(scale) - e_ref, 0) + code_shift<FMT>(), -126)));
        };
        auto scales_of = [&](int id) {
          if (id < 0) return make_float2(1.f, 1.f);
          const int64_t at = static_cast<int64_t>(id) * p.heads + h;
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
          const int row = mine ? static_cast<int>((static_cast<int64_t>(id0) * p.heads + h) * p.block) : 0;
          const int from = k * ppt + (lane & 7) * 16 / p.block;
          const float a = __shfl_sync(0xffffffffu, sc0.x, from), v = __shfl_sync(0xffffffffu, sc0.y, from);
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            if (i > 0) wait(&stg_empty[hh], i - 1, 73);
            if (ok) {
              if (lane == 0 && valid) mbar_expect_tx(&stg_full[hh], static_cast<uint32_t>(pbytes) * __popc(valid));
              if (hh == 0 && lane < 8) {
                const __half2 rk = ratio(a, ke), rv = ratio(v, ve);
                ratios[(i & 7) * 8 + lane] = make_uint2(*reinterpret_cast<const uint32_t*>(&rk), *reinterpret_cast<const uint32_t*>(&rv));
                if (general) {
                  const float vm = v > 0.f ? scale_mantissa(v) : 1.f;   // (0: the codes' multiplier is as good as 0)
                  meta[(i & 7) * 8 + lane] = make_float4(scale_mantissa(a), log2f(vm), 1.f / vm, 0.f);
                }
              }
              __syncwarp();
              if (mine)
                tma_load_2d(smem + C::kStgOff + hh * C::kStg + (lane - k * ppt) * pbytes, hh ? &vmap : &kmap, 0, row,
                            &stg_full[hh]);
              __syncwarp();
              if (lane == 0) mbar_arrive(&stg_full[hh]);
            }
          }
        }
      }
      // (in the normal course the converters have waited for every copy)
      if (!ok && i > 0)
        for (int h = 0; h < 2; ++h) mbar_wait(&stg_full[h], static_cast<uint32_t>(i - 1) & 1u);
    } else if (warp == kPlan) {
      // ---------------- the plan, and the scales of each segment's pages
      const int ppt = kPromptTile / p.block;
      PromptWalk walk;
      walk.u = unit_begin(blockIdx.x, start.U, start.P);
      walk.end = unit_begin(blockIdx.x + 1, start.U, start.P);
      walk.b = start.b;
      walk.base = start.base;
      walk.load(p);
      walk.find();
      const long long ubeg = walk.u;
      int i = 0;
      bool more = true;
      for (int seg = 0; more && ok; ++seg) {
        wait(&seg_empty[seg & 3], (seg >> 2) + 1, 74);
        Segment s;
        more = walk.next(p, s, ubeg);
        if (more) {
          // (the walk may be at the next sequence already)
          const PageRun run = read_pages(SeqInfo{s.start, s.kv - s.past, s.kv}, p.block, p.window);
          const int from = max(run.first, s.tile * ppt), to = min(run.first + run.n, (s.tile + s.units) * ppt);
          int ke = -126, ve = -126;
          bool mantissas = false;
#pragma unroll 4
          for (int pg = from + lane; pg < to; pg += 32) {
            const int id = page_block(p.seqs, s.b, pg, p.num_blocks);
            const int64_t at = static_cast<int64_t>(max(id, 0)) * p.heads + s.h;
            const float a = p.ks[at], b = p.vs[at];
            if (id < 0) continue;
            ke = max(ke, scale_exponent(a)), ve = max(ve, scale_exponent(b));
            mantissas |= scale_mantissa(a) != 1.f || scale_mantissa(b) != 1.f;
          }
          __syncwarp();
          s.ke = __reduce_max_sync(0xffffffffu, ke);
          s.ve = __reduce_max_sync(0xffffffffu, ve);
          s.general = __any_sync(0xffffffffu, mantissas);
          s.meta = i & 7;
          i += s.units;
          if (lane == 0 && s.slot >= 0 && (s.slot & 1)) {   // the CTA's last item, which others go on with
            const long long last = walk.base + walk.h * walk.w.per_head + walk.at + walk.nt - 1;
            join_items<D>(p, gridDim.x)[blockIdx.x] = {cta_of_unit(last, start.U, start.P), s.start, s.rows, s.row0, s.h, {}};
          }
        }
        if (lane == 0) {
          segs[seg & 3] = s;
          mbar_arrive(&seg_full[seg & 3]);
        }
        __syncwarp();
      }
    }
  }
  __syncwarp();

  tc_fence_before();
  cta_sync();
  tc_fence_after();
  if (warp == kIssue0) tmem_dealloc(tmem, 512);
}

constexpr int kEl = 16;
// Joins the partials of the items that several CTAs share.  Block x has the
// item that CTA x begins, and CTAs up to `last` go on with, in their order;
// block y has kEl elements of its rows, a thread a row.  It runs while nothing
// else does, so its time is latency: it finds its item written down, and the
// loads of kWide partials are under way together.
template <int D>
__global__ void __launch_bounds__(kPromptRows) k_kv8_join(const AttnParams p, int ctas) {
  constexpr int kWide = 2;
  pdl_wait();   // every block: the kernels after this one must find the one before it done
  const int c = blockIdx.x;
  const JoinItem* at = join_items<D>(p, ctas) + c;
  const int4 it = __ldcg(reinterpret_cast<const int4*>(at));   // last, start, rows, row0
  const int h = __ldcg(&at->h);
  const int r = threadIdx.x, row = it.w + r;
  if (it.x < 0 || row >= it.z) return;
  const int tok = row / p.group, hd = h * p.group + row - tok * p.group;
  const int64_t tk = static_cast<int64_t>(it.y) + tok;
  constexpr size_t kSlot = PrCfg<D>::kSlot;
  float mx = -INFINITY, sum = 0.f, o[kEl];
#pragma unroll
  for (int k = 0; k < kEl; ++k) o[k] = 0.f;
#pragma unroll 1
  for (int cc = c; cc <= it.x; cc += kWide) {
    float m[kWide], l[kWide], v[kWide][kEl];
#pragma unroll
    for (int j = 0; j < kWide; ++j) {
      const float* sl = p.part + static_cast<size_t>(2 * min(cc + j, it.x) + (cc + j == c ? 1 : 0)) * kSlot + r;
      m[j] = cc + j <= it.x ? __ldcg(sl + D * kPromptRows) : -INFINITY;
      l[j] = __ldcg(sl + (D + 1) * kPromptRows);
#pragma unroll
      for (int k = 0; k < kEl; ++k)   // element e lies in column e % 4 D/4 + e / 4
        v[j][k] = __ldcg(sl + ((k & 3) * (D / 4) + kEl / 4 * blockIdx.y + (k >> 2)) * kPromptRows);
    }
    float top = mx;
#pragma unroll
    for (int j = 0; j < kWide; ++j) top = fmaxf(top, m[j]);
    const float ref = top == -INFINITY ? 0.f : top, f = exp2_approx(mx - ref);
    mx = top;
    sum *= f;
#pragma unroll
    for (int k = 0; k < kEl; ++k) o[k] *= f;
#pragma unroll
    for (int j = 0; j < kWide; ++j) {
      const float g = exp2_approx(m[j] - ref);
      sum = fmaf(g, l[j], sum);
#pragma unroll
      for (int k = 0; k < kEl; ++k) o[k] = fmaf(g, v[j][k], o[k]);
    }
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  uint32_t v[kEl / 2];
#pragma unroll
  for (int k = 0; k < kEl / 2; ++k) {
    const __nv_bfloat162 z = __floats2bfloat162_rn(o[2 * k] * inv, o[2 * k + 1] * inv);
    v[k] = *reinterpret_cast<const uint32_t*>(&z);
  }
  uint4* dst = reinterpret_cast<uint4*>(p.out + tk * p.os + static_cast<int64_t>(hd) * D + kEl * blockIdx.y);
#pragma unroll
  for (int k = 0; k < kEl / 8; ++k) dst[k] = make_uint4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
  if (blockIdx.y == 0 && p.lse) p.lse[tk * p.Hq + hd] = sum == 0.f ? -INFINITY : (mx + log2f(sum)) * kLn2;
}

template <int FMT, int D>
int launch(const CUtensorMap& km, const CUtensorMap& vm, const AttnParams& p, cudaStream_t s) {
  using C = PrCfg<D>;
  static bool attr_done[64] = {false};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return FL_ERR_CUDA;
  if (dev >= 64 || !attr_done[dev]) {
    cudaFuncAttributes fa;   // the roles' register counts add up to the launch's
    if (cudaFuncGetAttributes(&fa, k_kv8_prompt<FMT, D>) != cudaSuccess || fa.numRegs != kRegs ||
        cudaFuncSetAttribute(k_kv8_prompt<FMT, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem) != cudaSuccess)
      return FL_ERR_CUDA;
    if (dev < 64) attr_done[dev] = true;
  }
  const int ctas = flh::sm_count();
  const int e = flh::launch_early(k_kv8_prompt<FMT, D>, ctas, kPrThreads, C::kSmem, s, km, vm, p);
  if (e != FL_OK || ctas < 2) return e;
  return flh::launch_early(k_kv8_join<D>, dim3(ctas - 1, D / kEl), kPromptRows, 0, s, p, ctas);
}

}  // namespace

namespace flkv {

size_t prompt_scratch(int head_dim) {
  return flh::sm_count() * (2 * static_cast<size_t>(kPromptRows) * (head_dim + 2) * 4 + sizeof(JoinItem));
}

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
