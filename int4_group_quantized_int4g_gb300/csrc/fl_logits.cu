// From logits to the next token: penalties for tokens that have come, biases,
// temperature, a mask of allowed tokens, then the largest, the row's log sum exp
// and the token's log-probability, in one pass over the logits.
//
// A CTA owns a run of a row's vocabulary, whose logits come into shared memory by
// one bulk copy, so that the bytes in flight do not depend on registers.
// Meanwhile it counts the row's history: one word a token of its run, how often it
// stands in the answer, the top bit for the prompt; whoever counts a token first
// puts it on a list.  Every CTA of a row reads all of its history, out of L2, and
// keeps what falls into its run; where that is much, a kernel before puts the history in
// the order of the runs, while the logits are already on their way (512 rows of 128003
// with 2000 entries 108 us, not 116, with 7000 112 and 166, with 16000 127 and 277).  Then
// the listed tokens, and those that a bias names, are changed in shared memory, a thread
// a token: one in a hundred has a penalty, but two of three warps meet one, so doing it
// on the way through the run cost 80 instructions a logit (512 rows of 128003: 261 us, and
// 161 with this change alone).
// Last the run passes through registers once: temperature, mask, the store, and a
// running maximum and sum of exp (x - max) a thread.  The runs' results are joined in
// their order, by the row's last CTA, or, with many CTAs, by a kernel of its own: a CTA
// that takes a ticket waits until its stores are seen (512 rows of 128003, unsorted, 116
// us, not 125; of few CTAs the second launch would cost the host more).  Every step of the rules is
// one fp32 rounding, so that equal logits stay equal and ties are the formula's.  Bound
// by HBM, the logits in and fp32 out, where there is little to look up (512 rows of 128003
// without rules 82 us, 6.4 TB/s), else by instructions: with histories of 1000 to 2000
// entries and 20 biases a row 107 us.
#include <type_traits>

#include "fl_common.cuh"

using namespace fl;

namespace {

constexpr int kLead = 32;                      // room before a run's first whole vector
constexpr int kRowsMax = kTicketTiles * kTicketWarps;   // tickets: rows of one launch
constexpr int kRunMin = 1024, kRunMax = 16384;
constexpr int kThreads = 256;                  // with short histories
constexpr int kJoinThreads = 64;
// A history of 1024 to 23040 entries (48 KB and counts of 16 bits hold them) is sorted by
// run where a row's CTAs, kApart an SM or more, would read 65536 entries an SM otherwise:
// there that is as much as the third launch costs the host.  512 rows of 128003 with 500
// entries 104 us unsorted, 105 sorted, with 1000 108 and 107, with 2000 116 and 108; 128
// rows with 1000 33 and 34, with 2000 36 and 34.  Fewer rows would gain in a captured
// graph alone: 48 rows with 4000 20 and 18 us of kernels, but 22 and 25 a call; 48 of
// 151655 with 4100, a grammar and biases 24 and 21, but 24 and 30.
constexpr int kSortThreads = 512;              // as many runs at most are sorted by
constexpr int kSortLeast = 1024, kSortMost = 23040;
constexpr long long kSortWork = 65536;
constexpr int kSortRows = 8192;                // rows of a launch then,
constexpr int kSortRoom = 1 << 23;             // and entries of all of them
// CTAs for each SM from which on a kernel of its own joins the runs: 64 rows of 128003
// (2048 CTAs) 21.2 us without, 20.1 with it, but 23.0 and 25.6 a call; 100 rows 29.9 and
// 28.6, and the same a call.
constexpr int kApart = 16;
constexpr int kRunBytes = 40960, kRunBytesLong = 81920;   // shared memory of a run, with short and long histories
constexpr int kRunBytesRow = 61440;            // of one that is the whole row

struct Partial {
  float top, sum;
  int index, pad;
};

struct LogitsParams {
  const void* x;
  float* out;
  int32_t* token;
  float* lse;
  float* logprob;
  Partial* part;      // [row][run]
  int32_t* cnt;       // [row]
  int32_t* status;
  int64_t xs, os;
  fl_logits_rules r;
  int V, run, runs;   // a run: tokens after the row's first 16-byte boundary
  int vec_out, vec_h;
  int apart;          // a kernel of its own joins the runs
  uint16_t* sorted;   // [row][sorted_stride] history by run, or NULL: place in the run's shared memory, top bit: prompt
  int32_t* begin;     // [row][runs + 1] where in it each run's entries begin
  int sorted_stride, shift;   // run is 1 << shift
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float exp_of(float d) { return ex2(d * 1.44269504f); }   // exp(d), d <= 0, relative to within |d| 2^-24 + 2^-22

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<const uint64_t&>(a)), "l"(reinterpret_cast<const uint64_t&>(b)));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<const uint64_t&>(a)), "l"(reinterpret_cast<const uint64_t&>(b)));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {   // (a NaN loses)
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// A maximum, the first index that has it, and the sum of exp(x - maximum) of all others:
// where one token has nearly all of the probability, its logarithm is this sum, and would
// be lost in 1 + sum.
struct Best {
  float top, sum;
  int index;
  __device__ __forceinline__ float all() const { return top > -INFINITY ? sum + 1.f : sum; }   // (the maximum's own with it)
  __device__ __forceinline__ void join(const Best& o) {
    const bool other = o.top > top || (o.top == top && static_cast<unsigned>(o.index) < static_cast<unsigned>(index));
    const float t = fmaxf(top, o.top), base = t == -INFINITY ? 0.f : t;
    sum = other ? o.sum + all() * exp_of(top - base) : sum + o.all() * exp_of(o.top - base);
    if (other) index = o.index;
    top = t;
  }
  __device__ __forceinline__ void join_warp() {
    float t = top;
#pragma unroll
    for (int d = 16; d; d >>= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, d));
    const float base = t == -INFINITY ? 0.f : t;
    const unsigned first = __reduce_min_sync(0xffffffffu, top == t ? static_cast<unsigned>(index) : 0xffffffffu);
    if (top != t || static_cast<unsigned>(index) != first) sum = all() * exp_of(top - base);
#pragma unroll
    for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);   // (the same sum in every lane)
    index = static_cast<int>(first);
    top = t;
  }
};

// Tokens of a row before its first 16-byte boundary: run 0 begins there, and holds them too.
template <typename Raw>
__device__ __forceinline__ int row_head(const void* row, int V) {
  return min(static_cast<int>((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / static_cast<int>(sizeof(Raw)), V);
}

// The row's results from `all` of it.
__device__ __forceinline__ void write_row(const LogitsParams& p, uint32_t b, const Best& all) {
  const bool none = all.top == -INFINITY;
  const float l = none ? (all.sum == 0.f ? INFINITY : NAN) : all.top == INFINITY ? NAN : log1pf(all.sum);
  p.token[b] = all.index;
  if (p.lse) p.lse[b] = none ? -l : all.top + l;
  if (p.logprob) p.logprob[b] = -l;
}
// Joins the row's runs, with T threads, and writes the row's results.
template <int T>
__device__ __forceinline__ void join_runs(const LogitsParams& p, uint32_t b, Best* warps) {
  const int tid = threadIdx.x;
  Best best = {-INFINITY, 0.f, -1};
  for (int i = tid; i < p.runs; i += T) {
    const float4 f = __ldcg(reinterpret_cast<const float4*>(p.part + static_cast<int64_t>(b) * p.runs + i));
    best.join(Best{f.x, f.y, __float_as_int(f.z)});
  }
  best.join_warp();
  if ((tid & 31) == 0) warps[tid >> 5] = best;
  __syncthreads();
  if (tid < 32) {
    best = tid < T / 32 ? warps[tid] : Best{-INFINITY, 0.f, -1};
    best.join_warp();
    if (tid == 0) write_row(p, b, best);
  }
}

// Shared memory of a run of `room` tokens: the logits; for history or biases a
// word a token (its count, 16 bits with fp32 logits and few entries; with bf16
// logits the changed value); a list of history's tokens, for a quarter of them; a
// bit a token for those that a bias names, and with bf16 for changed ones.
__host__ __device__ constexpr int word_bytes(bool bf16, bool history, bool biases, bool many) {
  return history ? (bf16 || many ? 4 : 2) : (bf16 && biases ? 4 : 0);
}
__host__ __device__ constexpr int run_bytes(int room, bool bf16, bool history, bool biases, bool many) {
  return room * ((bf16 ? 2 : 4) + word_bytes(bf16, history, biases, many)) + (history ? room / 2 : 0) + room / 32 * 8 + 16;
}

template <bool BF16, bool LONG>
__global__ void __launch_bounds__(LONG ? 1024 : kThreads) k_logits(const LogitsParams p) {
  constexpr int W = BF16 ? 8 : 4;    // tokens of a 16-byte vector
  constexpr int T = LONG ? 1024 : kThreads;
  constexpr bool HALF = !BF16 && !LONG;   // counts of 16 bits
  using Raw = std::conditional_t<BF16, uint16_t, float>;
  extern __shared__ uint4 raw[];
  __shared__ Best warps[T / 32];
  __shared__ int again, finish, listed;
  __shared__ uint64_t landed;
  const int tid = threadIdx.x;
  const uint32_t b = blockIdx.x / static_cast<uint32_t>(p.runs), run = blockIdx.x - b * p.runs;
  const fl_logits_rules& r = p.r;
  const int room = p.run + kLead;
  const bool counts = r.history != nullptr, biases = r.bias_ids != nullptr;
  Raw* x = reinterpret_cast<Raw*>(raw);
  uint32_t* word = reinterpret_cast<uint32_t*>(x + room);
  uint32_t* named = word + room * word_bytes(BF16, counts, biases, LONG) / 4;   // bits: a bias names the token
  uint32_t* changed = named + room / 32 + 1;                          // bits: word holds the token's value
  uint16_t* list = reinterpret_cast<uint16_t*>(changed + room / 32 + 1);
  if (tid == 0) {
    again = listed = 0;
    mbar_init(&landed, 1);
    fence_mbar_init();
  }
  if (counts)
    for (int i = tid; i < room / (HALF ? 8 : 4); i += T) reinterpret_cast<uint4*>(word)[i] = make_uint4(0, 0, 0, 0);
  if (BF16 || biases)
    for (int i = tid; i < 2 * (room / 32 + 1); i += T) named[i] = 0;

  // (after k_logits_sort, which has waited for all kernels before it, the logits are there)
  if (LONG || !p.sorted) pdl_wait();
  const uint8_t* row = static_cast<const uint8_t*>(p.x) + static_cast<int64_t>(b) * p.xs * (BF16 ? 2 : 4);
  float* out = p.out ? p.out + static_cast<int64_t>(b) * p.os : nullptr;
  // the row's first token on 16 bytes; a run starts there or whole runs behind
  const int head = row_head<Raw>(row, p.V);
  const int64_t first = head + static_cast<int64_t>(run) * p.run;
  const int start = static_cast<int>(min(first, static_cast<int64_t>(p.V)));
  const int lo = run == 0 ? 0 : start, hi = static_cast<int>(min(first + p.run, static_cast<int64_t>(p.V)));
  const int base = start - kLead;    // token 0 of shared memory
  const int nvec = (hi - start) / W, tail = start + nvec * W;
  if (tid == 0 && nvec) {
    mbar_arrive_expect_tx(&landed, nvec * 16);
    bulk_g2s(x + kLead, row + static_cast<int64_t>(start) * (BF16 ? 2 : 4), nvec * 16, &landed);
  }
  if (!LONG && p.sorted) pdl_wait();
  pdl_launch_dependents();
  // the history's entries, four at a time; the first are on their way before the
  // lengths are known (lists are history_max long whatever of them counts)
  constexpr int kAhead = LONG ? 2 : 512 / kThreads;
  int4 ahead[kAhead];
  int n = 0, prompt = 0;
  const int32_t* h = r.history + static_cast<int64_t>(b) * r.history_stride;
  auto fetch = [&](int i) {
    int4 f = make_int4(-1, -1, -1, -1);
    if (p.vec_h && 4 * i + 4 <= r.history_max) return __ldg(reinterpret_cast<const int4*>(h) + i);
    if (4 * i >= r.history_max) return f;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (4 * i + e < r.history_max) (&f.x)[e] = __ldg(h + 4 * i + e);
    return f;
  };
  if (counts && (LONG || !p.sorted)) {
    n = min(max(__ldg(r.history_lens + b), 0), r.history_max);
    prompt = r.prompt_lens ? max(__ldg(r.prompt_lens + b), 0) : 0;
#pragma unroll
    for (int k = 0; k < kAhead; ++k) ahead[k] = fetch(tid + k * T);
  }
  // the few tokens before the first vector and after the last
  const int few = (start - lo) + (hi - tail);
  auto few_at = [&](int i) { return i < start - lo ? lo + i : tail + (i - (start - lo)); };
  if (tid < few) x[few_at(tid) - base] = reinterpret_cast<const volatile Raw*>(row)[few_at(tid)];
  __syncthreads();

  // an entry of a short history: counts it, and lists its token
  auto count = [&](int i1, bool asked) {
    const int shift = HALF ? (i1 & 1) * 16 : 0;
    uint32_t* w = word + (HALF ? i1 >> 1 : i1);
    const uint32_t old = asked ? atomicOr(w, HALF ? 0x8000u << shift : 0x80000000u) : atomicAdd(w, 1u << shift);
    if ((HALF ? old >> shift & 0xffffu : old) == 0) {
      const int to = atomicAdd(&listed, 1);
      if (to < room / 4) list[to] = static_cast<uint16_t>(i1);
    }
  };
  if (!LONG && p.sorted) {
    const int32_t* begin = p.begin + static_cast<int64_t>(b) * (p.runs + 1) + run;
    const uint16_t* ids = p.sorted + static_cast<int64_t>(b) * p.sorted_stride;
    const int end = __ldcg(begin + 1);
    for (int i = __ldcg(begin) + tid; i < end; i += T) {
      const uint32_t id = __ldcg(ids + i);
      count(id & 0x7fff, id >> 15);
    }
  } else if (counts) {
    const uint32_t width = hi - lo;
    // four entries of a long history, all of the prompt or all of the answer: an
    // operation in shared memory for each, without a branch
    const uint32_t first_word = smem_u32(word + (lo - base));
    auto four = [&](const int4& f, auto answer) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t off = static_cast<uint32_t>((&f.x)[e] - lo);
        if constexpr (decltype(answer)::value)
          asm volatile("{\n\t.reg .pred p;\n\tsetp.lt.u32 p, %0, %1;\n\t@p red.shared.add.u32 [%2], 1;\n\t}" ::"r"(off), "r"(width),
                       "r"(first_word + 4 * off)
                       : "memory");
        else
          asm volatile("{\n\t.reg .pred p;\n\tsetp.lt.u32 p, %0, %1;\n\t@p red.shared.or.b32 [%2], %3;\n\t}" ::"r"(off), "r"(width),
                       "r"(first_word + 4 * off), "r"(0x80000000u)
                       : "memory");
      }
    };
    for (int i = tid; 4 * i < n; i += kAhead * T) {
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        if constexpr (LONG) {
          const int at = 4 * (i + k * T);
          if (at >= prompt && at + 4 <= n) {
            four(ahead[k], std::true_type());
            continue;
          }
          if (at + 4 <= min(prompt, n)) {
            four(ahead[k], std::false_type());
            continue;
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int id = (&ahead[k].x)[e], at = 4 * (i + k * T) + e;
          if (static_cast<uint32_t>(id - lo) < width && at < n) {
            if constexpr (LONG) {
              uint32_t* w = word + (id - base);
              if (at < prompt)
                atomicOr(w, 0x80000000u);
              else
                atomicAdd(w, 1u);
            } else {
              count(id - base, at < prompt);
            }
          }
        }
      }
      if (4 * (i + kAhead * T) < n) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k) ahead[k] = fetch(i + (kAhead + k) * T);
      }
    }
  }
  int bias_lo = 0, bias_hi = 0;
  if (biases) {
    bias_lo = min(max(r.bias_offsets[b], 0), r.bias_count);
    bias_hi = min(max(r.bias_offsets[b + 1], bias_lo), r.bias_count);
    for (int i = bias_lo + tid; i < bias_hi; i += T) {
      const int id = __ldg(r.bias_ids + i);
      if (id >= lo && id < hi) {
        const uint32_t bit = 1u << ((id - base) & 31);
        if (atomicOr(named + ((id - base) >> 5), bit) & bit) again = 1;
      }
    }
  }
  if (tid == 0 && nvec && !mbar_wait(&landed, 0)) set_status(p.status, FL_ERR_TIMEOUT, 60);
  __syncthreads();   // (counted, listed, landed)

  auto value = [&](int i) {   // of token base + i
    if constexpr (BF16) {
      if (changed[i >> 5] >> (i & 31) & 1) return __uint_as_float(word[i]);
      return __uint_as_float(static_cast<uint32_t>(x[i]) << 16);
    } else {
      return x[i];
    }
  };
  auto change = [&](int i, float v) {
    if constexpr (BF16) {
      word[i] = __float_as_uint(v);
      atomicOr(changed + (i >> 5), 1u << (i & 31));
    } else {
      x[i] = v;
    }
  };
  if (counts) {
    const float rep = r.repetition ? r.repetition[b] : 1.f, freq = r.frequency ? r.frequency[b] : 0.f;
    const float pres = r.presence ? r.presence[b] : 0.f;
    auto penalise = [&](int i) {
      const uint32_t c = HALF ? word[i >> 1] >> ((i & 1) * 16) & 0x7fffu : word[i] & 0x7fffffffu;
      float v = value(i);
      if (r.repetition) v = v > 0.f ? __fdiv_rn(v, rep) : __fmul_rn(v, rep);
      if (c) {
        if (r.frequency) v = __fsub_rn(v, __fmul_rn(freq, static_cast<float>(c)));
        if (r.presence) v = __fsub_rn(v, pres);
      }
      change(i, v);
    };
    // a long history comes back to the same tokens again and again: there the counts
    // are looked through for the tokens, not asked for with every entry
    if (LONG || listed > room / 4) {
      __syncthreads();
      if (tid == 0) listed = 0;
      __syncthreads();
      for (int i = tid; i < room; i += T) {
        if (!(HALF ? word[i >> 1] >> ((i & 1) * 16) & 0xffffu : word[i])) continue;
        const int at = atomicAdd(&listed, 1);
        if (at < room / 4)
          list[at] = static_cast<uint16_t>(i);
        else   // (the list is full)
          penalise(i);
      }
      __syncthreads();
    }
    for (int j = tid; j < min(listed, room / 4); j += T) penalise(list[j]);
    __syncthreads();
  }
  if (biases) {
    // a token that is named again gets its biases in list order, from one thread (which
    // looks through all of the list: 48 rows of 128003 with 4000 biases 272 us, not 19)
    const bool several = again != 0;
    for (int i = several ? bias_lo : bias_lo + tid; i < bias_hi; i += several ? 1 : T) {
      const int id = __ldg(r.bias_ids + i);
      if (id >= lo && id < hi && (!several || id % T == tid)) change(id - base, __fadd_rn(value(id - base), __ldg(r.bias + i)));
    }
    __syncthreads();
  }

  float inv = 1.f;
  if (r.temperature) {
    const float t = r.temperature[b];
    inv = t > 0.f ? __fdiv_rn(1.f, t) : 1.f;
  }
  const uint32_t* mask = r.allowed ? reinterpret_cast<const uint32_t*>(r.allowed) + static_cast<int64_t>(b) * r.allowed_stride : nullptr;
  Best best = {-INFINITY, 0.f, -1};
  float zero = 0.f;   // what is added before exp: the maximum's negative, 0 without one
  auto one = [&](int v) {   // a token outside the vectors
    float f = __fmul_rn(value(v - base), inv);
    if (mask && !(__ldg(mask + (v >> 5)) >> (v & 31) & 1)) f = -INFINITY;
    if (out) out[v] = f;
    best.join(Best{f == f ? f : -INFINITY, f == f ? 0.f : f, f > -INFINITY ? v : -1});
  };
  // N vectors, T apart.  What a call has not is decided once, not with every vector
  auto vectors = [&](int j, auto has_out, auto has_mask, auto count) {
    constexpr int N = decltype(count)::value;
    float f[N * W];
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int at = kLead + (j + n * T) * W, v = base + at;
      const uint4 u = *reinterpret_cast<const uint4*>(x + at);
      float* g = f + n * W;
      if constexpr (BF16) {
#pragma unroll
        for (int e = 0; e < W; ++e) g[e] = __uint_as_float(e & 1 ? (&u.x)[e / 2] & 0xffff0000u : (&u.x)[e / 2] << 16);
        if (counts || biases) {
          const uint32_t bits = reinterpret_cast<const uint8_t*>(changed)[at / 8];
          if (bits) {
#pragma unroll
            for (int e = 0; e < W; ++e)
              if (bits >> e & 1) g[e] = __uint_as_float(word[at + e]);
          }
        }
      } else {
#pragma unroll
        for (int e = 0; e < W; ++e) g[e] = __uint_as_float((&u.x)[e]);
      }
#pragma unroll
      for (int e = 0; e < W; e += 2) {
        const float2 h = mul2(make_float2(g[e], g[e + 1]), make_float2(inv, inv));
        g[e] = h.x, g[e + 1] = h.y;
      }
      if constexpr (decltype(has_mask)::value) {
        const uint32_t w0 = __ldg(mask + (v >> 5));
        const uint32_t w1 = (v & 31) + W > 32 ? __ldg(mask + (v >> 5) + 1) : 0;
        const uint32_t bits = __funnelshift_r(w0, w1, v & 31);
#pragma unroll
        for (int e = 0; e < W; ++e)
          if (!(bits >> e & 1)) g[e] = -INFINITY;
      }
      if constexpr (decltype(has_out)::value) {
        if (p.vec_out) {
#pragma unroll
          for (int q = 0; q < W / 4; ++q)
            __stcs(reinterpret_cast<float4*>(out + v) + q, make_float4(g[4 * q], g[4 * q + 1], g[4 * q + 2], g[4 * q + 3]));
        } else {
#pragma unroll
          for (int e = 0; e < W; ++e) out[v + e] = g[e];
        }
      }
    }
    float top = max3(f[0], f[1], f[2]);
#pragma unroll
    for (int e = 3; e + 1 < N * W; e += 2) top = max3(top, f[e], f[e + 1]);
    top = fmaxf(top, f[N * W - 1]);
    if (top > best.top) {
      best.sum = best.all() * exp_of(best.top - top);
      best.top = top;
      zero = -top;   // (not -inf: it is above another)
      int at = 0;
#pragma unroll
      for (int e = N * W - 1; e >= 0; --e)
        if (f[e] == top) at = e;
#pragma unroll
      for (int e = 0; e < N * W; ++e)
        if (at == e) f[e] = -INFINITY;   // (not in the sum)
      best.index = base + kLead + (j + at / W * T) * W + at % W;
    }
    float2 sum = make_float2(0.f, 0.f);
#pragma unroll
    for (int e = 0; e < N * W; e += 2) {
      const float2 d = mul2(add2(make_float2(f[e], f[e + 1]), make_float2(zero, zero)), make_float2(1.44269504f, 1.44269504f));
      sum = add2(sum, make_float2(ex2(d.x), ex2(d.y)));
    }
    best.sum += sum.x + sum.y;
  };
  auto all = [&](auto has_out, auto has_mask) {
    int j = tid;
    if constexpr (!BF16) {
#pragma unroll 1
      for (; j + T < nvec; j += 2 * T) vectors(j, has_out, has_mask, std::integral_constant<int, 2>());
    }
    for (; j < nvec; j += T) vectors(j, has_out, has_mask, std::integral_constant<int, 1>());
  };
  // a thread's tokens in ascending order: before the vectors, these, after them
  if (tid < start - lo) one(lo + tid);
  zero = best.top == -INFINITY ? 0.f : -best.top;
  using Yes = std::true_type;
  using No = std::false_type;
  if (out) {
    if (mask)
      all(Yes(), Yes());
    else
      all(Yes(), No());
  } else if (mask) {
    all(No(), Yes());
  } else {
    all(No(), No());
  }
  if (tid < hi - tail) one(tail + tid);

  best.join_warp();
  if ((tid & 31) == 0) warps[tid >> 5] = best;
  __syncthreads();
  if (p.apart && tid >= 32) return;
  if (tid < 32) {
    best = tid < T / 32 ? warps[tid] : Best{-INFINITY, 0.f, -1};
    best.join_warp();
    if (tid == 0) {
      finish = 0;
      if (p.runs == 1) {
        write_row(p, b, best);
      } else {
        __stcg(reinterpret_cast<float4*>(p.part + static_cast<int64_t>(b) * p.runs + run),
               make_float4(best.top, best.sum, __int_as_float(best.index), 0.f));
        if (!p.apart) {
          finish = atom_add_acq_rel_gpu(p.cnt + b, 1) == p.runs - 1;
          if (finish) p.cnt[b] = 0;
        }
      }
    }
  }
  if (p.apart) return;
  __syncthreads();
  if (finish) join_runs<T>(p, b, warps);
}

// Puts the history of a row (a CTA's) in the order of the runs, each entry as what a run's
// CTA makes of it.
template <typename Raw>
__global__ void __launch_bounds__(kSortThreads) k_logits_sort(const LogitsParams p) {
  extern __shared__ uint4 raw[];
  __shared__ int at[kSortThreads], sums[kSortThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, b = blockIdx.x;
  at[tid] = 0;
  pdl_wait();
  pdl_launch_dependents();   // (after the wait: k_logits, started now, finds the logits)
  const fl_logits_rules& r = p.r;
  const int head = row_head<Raw>(static_cast<const Raw*>(p.x) + b * p.xs, p.V);
  const int n = min(max(r.history_lens[b], 0), r.history_max), prompt = r.prompt_lens ? r.prompt_lens[b] : 0;
  const int32_t* h = r.history + b * r.history_stride;
  auto fetch = [&](int i) {
    int4 f = make_int4(-1, -1, -1, -1);
    if (p.vec_h && i + 4 <= r.history_max) return *reinterpret_cast<const int4*>(h + i);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (i + e < r.history_max) (&f.x)[e] = h[i + e];
    return f;
  };
  const int4 first = fetch(4 * tid);
  auto each = [&](auto take) {   // (run, entry of the sorted list)
    for (int i = 4 * tid; i < n; i += 4 * kSortThreads) {
      const int4 f = i == 4 * tid ? first : fetch(i);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int id = (&f.x)[e];
        if (i + e >= n || id < 0 || id >= p.V) continue;
        const int run = max(id - head, 0) >> p.shift;
        // (its shared memory holds the tokens from head + run's first less kLead on)
        take(run, static_cast<uint16_t>(id - head - (run << p.shift) + kLead) | (i + e < prompt ? 0x8000u : 0u));
      }
    }
  };
  __syncthreads();
  each([&](int run, uint32_t) { atomicAdd(&at[run], 1); });
  __syncthreads();
  const int v = at[tid];
  int inc = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, inc, d);
    if (lane >= d) inc += u;
  }
  if (lane == 31) sums[tid >> 5] = inc;
  __syncthreads();
  for (int w = 0; w < tid >> 5; ++w) inc += sums[w];
  int32_t* begin = p.begin + static_cast<int64_t>(b) * (p.runs + 1);
  if (tid < p.runs) begin[tid + 1] = inc;
  if (tid == 0) begin[0] = 0;
  at[tid] = inc - v;
  __syncthreads();
  uint16_t* ids = reinterpret_cast<uint16_t*>(raw);
  each([&](int run, uint32_t id) { ids[atomicAdd(&at[run], 1)] = static_cast<uint16_t>(id); });
  __syncthreads();
  uint4* to = reinterpret_cast<uint4*>(p.sorted + static_cast<int64_t>(b) * p.sorted_stride);
  for (int i = tid; 8 * i < at[p.runs - 1]; i += kSortThreads) to[i] = raw[i];   // (whole vectors: the stride has room)
}

__global__ void __launch_bounds__(kJoinThreads) k_logits_join(const LogitsParams p) {
  __shared__ Best warps[kJoinThreads / 32];
  pdl_wait();
  pdl_launch_dependents();
  join_runs<kJoinThreads>(p, blockIdx.x, warps);
}

bool aligned(const void* p, int n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// Tokens of a run: the longest that fits its shared memory and still gives the
// GPU CTAs enough; short ones where rows are few.  Each of a row's CTAs reads all of
// its history: with a long one a CTA for two SMs is enough (12 rows of 32000 with 131000
// entries: 19 us with 96 CTAs, 27 with 192, which L2 feeds no faster).  With short ones
// five CTAs an SM are best (512 rows of 128003 108 us; runs of 8192, three an SM, 114; runs
// of 2048 156), but for a row that one run holds (2000 rows of 5000: 24 us, in two runs 28).
// From kLong entries on, by the width of the list, as the lengths are on the device: 1024
// threads.  With as many entries 12 rows of 32000 take 8.2 us with 256 threads and 9.0 with
// 1024 at 2000, 9.3 and 9.0 at 4100, 11.4 and 9.2 at 8192, 17.7 and 10.4 at 20000; 48 rows of
// 128003 18.7 and 28.5 at 4100, 23.6 and 29.4 at 8192, 30.0 and 31.5 at 12000, 40.5 and 33.8 at
// 20000.  A wide list with short lengths pays for that: 512 rows of 128003 with up to 2000
// entries take 107 us in lists of up to 23040, 229 in wider ones; one row 7.5 and 8.5.
constexpr int kLong = 8192;
int run_length(int B, int V, bool bf16, bool history, bool biases, bool many) {
  const long long want = (many ? 1ll : 8ll) * flh::sm_count() / 2;
  auto most = [&](int run) { return many ? kRunBytesLong : run >= V ? kRunBytesRow : kRunBytes; };
  int run = kRunMax;
  while (run > kRunMin && (run_bytes(run, bf16, history, biases, many) > most(run) || (V + run - 1ll) / run * B < want)) run /= 2;
  return run;
}
int run_shortest(int B, int V) {   // of all types and rules (long histories need fewer CTAs)
  const int a = run_length(B, V, false, true, true, false), b = run_length(B, V, true, true, true, false);
  const int c = run_length(B, V, false, true, true, true);
  return a < b ? (a < c ? a : c) : (b < c ? b : c);
}
int run_count(int V, int run) { return static_cast<int>((V + run - 1ll) / run); }

template <bool BF16, bool LONG>
int launch(const LogitsParams& p, int B, size_t smem, cudaStream_t s) {
  static bool ready[64] = {false};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 0 && dev < 64 && !ready[dev]) {
    if (cudaFuncSetAttribute(k_logits<BF16, LONG>, cudaFuncAttributeMaxDynamicSharedMemorySize, run_bytes(kRunMax + kLead, BF16, true, true, LONG)) != cudaSuccess) {
      cudaGetLastError();
      return FL_ERR_CUDA;
    }
    ready[dev] = true;
  }
  return flh::launch_early(k_logits<BF16, LONG>, dim3(static_cast<unsigned>(B) * p.runs), dim3(LONG ? 1024 : kThreads), smem, s, p);
}

// Whether rows of `out` would lie over rows of the logits, the logits themselves
// (the same place and stride, fp32) apart.
bool over(const void* x, int64_t xs, int size, const float* out, int64_t os, int B, int V) {
  if (x == out && size == 4 && xs == os) return false;
  return flh::rows_meet(x, xs * size, static_cast<uint64_t>(V) * size, B, out, os * 4, static_cast<uint64_t>(V) * 4, B);
}

// Workspace: the runs' results, where each run's entries of a sorted history begin, these.
struct LogitsLayout {
  size_t begin, sorted, bytes;
};
LogitsLayout layout(int B, int V) {
  const long long runs = run_count(V, run_shortest(B, V));
  auto up = [](size_t v) { return (v + 255) / 256 * 256; };
  LogitsLayout l;
  l.begin = up(kScratchOff + static_cast<size_t>(B < kRowsMax ? B : kRowsMax) * runs * sizeof(Partial));
  l.sorted = l.bytes = l.begin;
  if (B * runs > kApart * flh::sm_count()) {
    l.sorted = l.begin + up(static_cast<size_t>(B < kSortRows ? B : kSortRows) * ((runs < kSortThreads ? runs : kSortThreads) + 1) * 4);
    l.bytes = l.sorted + kSortRoom * 2;
  }
  return l;
}

bool logits_args(int B, int V) { return B >= 1 && V >= 1 && V < (1 << 30) && B <= (1 << 30); }

}  // namespace

extern "C" int fl_logits_process_workspace(int B, int V, size_t* out) {
  if (!out || !logits_args(B, V)) return FL_ERR_ARG;
  *out = layout(B, V).bytes;
  return FL_OK;
}

extern "C" int fl_logits_process(const void* logits, int64_t logits_stride, int type, int B, int V,
                                 const fl_logits_rules* rules, float* out, int64_t out_stride, int32_t* token, float* lse,
                                 float* logprob, void* ws, size_t ws_bytes, fl_stream_t stream) {
  if (!logits || !rules || !token || !ws || !logits_args(B, V) || (type != FL_OUT_BF16 && type != FL_OUT_FP32)) return FL_ERR_ARG;
  const bool bf16 = type == FL_OUT_BF16;
  const fl_logits_rules& r = *rules;
  if (logits_stride < V || (out && out_stride < V) || !flh::aligned16(ws) || !aligned(logits, bf16 ? 2 : 4)) return FL_ERR_ARG;
  const void* lists[] = {out, token, lse, logprob, r.history, r.history_lens, r.prompt_lens, r.repetition, r.frequency,
                         r.presence, r.bias_offsets, r.bias_ids, r.bias, r.allowed, r.temperature};
  for (const void* q : lists)
    if (!aligned(q, 4)) return FL_ERR_ARG;
  if (out && over(logits, logits_stride, bf16 ? 2 : 4, out, out_stride, B, V)) return FL_ERR_ARG;
  if (!r.history != !r.history_lens || (r.history && (r.history_max < 0 || r.history_max >= 1 << 30 || r.history_stride < r.history_max)))
    return FL_ERR_ARG;
  if (!r.history && (r.prompt_lens || r.repetition || r.frequency || r.presence)) return FL_ERR_ARG;
  if (!r.bias_offsets != !r.bias_ids || !r.bias_ids != !r.bias || (r.bias && r.bias_count < 0)) return FL_ERR_ARG;
  if (r.allowed && r.allowed_stride < (V + 31) / 32) return FL_ERR_ARG;
  const LogitsLayout l = layout(B, V);
  if (ws_bytes < l.bytes) return FL_ERR_WORKSPACE;

  LogitsParams p = {};
  p.xs = logits_stride, p.os = out_stride, p.r = r, p.V = V;
  bool many = r.history && r.history_max >= kLong;
  p.run = run_length(B, V, bf16, r.history, r.bias, false);
  p.runs = run_count(V, p.run);
  if (r.history && r.history_max >= kSortLeast && r.history_max <= kSortMost && p.runs > 1 && p.runs <= kSortThreads &&
      static_cast<long long>(B) * p.runs > kApart * flh::sm_count() &&
      static_cast<long long>(B) * p.runs * r.history_max > kSortWork * flh::sm_count()) {
    many = false;
    p.sorted = reinterpret_cast<uint16_t*>(static_cast<uint8_t*>(ws) + l.sorted);
    p.begin = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(ws) + l.begin);
    p.sorted_stride = (r.history_max + 7) / 8 * 8;
    while (1 << p.shift < p.run) ++p.shift;
  } else if (many) {
    p.run = run_length(B, V, bf16, r.history, r.bias, true);
    p.runs = run_count(V, p.run);
  }
  p.part = reinterpret_cast<Partial*>(static_cast<uint8_t*>(ws) + kScratchOff);
  p.cnt = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(ws) + kTicketOff);
  p.status = static_cast<int32_t*>(ws);
  p.vec_h = aligned(r.history, 16) && r.history_stride % 4 == 0;
  // a row's tokens on 16 bytes are so in both (rows shift both alike)
  const int64_t size = bf16 ? 2 : 4;
  const uintptr_t in0 = reinterpret_cast<uintptr_t>(logits) / size, out0 = reinterpret_cast<uintptr_t>(out) / 4;
  p.vec_out = out && (in0 - out0) % 4 == 0 && (logits_stride - out_stride) % 4 == 0;
  p.apart = p.runs > 1 && static_cast<long long>(B) * p.runs > kApart * flh::sm_count();
  const size_t smem = run_bytes(p.run + kLead, bf16, r.history, r.bias, many);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  for (int b = 0; b < B;) {
    int n = B - b < kRowsMax ? B - b : kRowsMax;
    const long long most = 0x7fffffffll / p.runs;
    if (n > most) n = static_cast<int>(most);
    if (p.sorted && n > kSortRows) n = kSortRows;
    if (p.sorted && n > kSortRoom / p.sorted_stride) n = kSortRoom / p.sorted_stride;
    LogitsParams q = p;
    q.x = static_cast<const uint8_t*>(logits) + static_cast<int64_t>(b) * logits_stride * size;
    q.out = out ? out + static_cast<int64_t>(b) * out_stride : nullptr;
    q.token = token + b, q.lse = lse ? lse + b : nullptr, q.logprob = logprob ? logprob + b : nullptr;
    auto row = [&](auto*& list, int64_t stride) { if (list) list += b * stride; };
    row(q.r.history, r.history_stride), row(q.r.history_lens, 1), row(q.r.prompt_lens, 1), row(q.r.repetition, 1);
    row(q.r.frequency, 1), row(q.r.presence, 1), row(q.r.bias_offsets, 1), row(q.r.allowed, r.allowed_stride), row(q.r.temperature, 1);
    if (p.sorted) {
      const int rs = flh::launch_early(bf16 ? k_logits_sort<uint16_t> : k_logits_sort<float>, dim3(n), dim3(kSortThreads), p.sorted_stride * 2, s, q);
      if (rs != FL_OK) return rs;
    }
    const int rc = many ? (bf16 ? launch<true, true>(q, n, smem, s) : launch<false, true>(q, n, smem, s))
                        : (bf16 ? launch<true, false>(q, n, smem, s) : launch<false, false>(q, n, smem, s));
    if (rc != FL_OK) return rc;
    if (p.apart) {
      const int rj = flh::launch_early(k_logits_join, dim3(n), dim3(kJoinThreads), 0, s, q);
      if (rj != FL_OK) return rj;
    }
    b += n;
  }
  return FL_OK;
}
