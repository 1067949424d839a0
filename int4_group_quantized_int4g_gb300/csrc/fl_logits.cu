// From logits to the next token: penalties for tokens that have come, biases,
// temperature, a mask of allowed tokens, then the largest, the row's log sum exp
// and the token's log-probability, in one pass over the logits.
//
// A CTA owns a run of a row's vocabulary.  It counts the row's history in shared
// memory, one word a token of its run: how often it stands in the answer, and the
// top bit for the prompt (so a word that is not 0 is a token that has been seen).
// Every CTA of a row reads all of its history, out of L2, and keeps what falls into
// its run.  Biases note the first entry of their list that names a token; entries
// that name one again are added in list order, by whoever owns the token.  Then the
// logits pass through registers once: the rules, the store, and a running maximum
// and sum of exp (x - max) a thread.  The runs' results are joined by the row's
// last CTA in their order.  Every step of the rules is one fp32 rounding, so that
// equal logits stay equal and ties are the formula's.  Bound by HBM: the logits in,
// fp32 out.
#include <limits>

#include "fl_common.cuh"

using namespace fl;

namespace {

constexpr int kLead = 8;                       // room before a run's first whole vector
constexpr int kRowsMax = kTicketTiles * kTicketWarps;   // tickets: rows of one launch
constexpr int kRunMin = 1024, kRunMax = 16384;

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
  int64_t xs, os;
  fl_logits_rules r;
  int V, run, runs;   // a run: tokens after the row's first 16-byte boundary
  int vec_x, vec_out, vec_h;
};

__device__ __forceinline__ float exp_of(float d) {   // exp(d), d <= 0
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(d * 1.44269504f));
  return y;
}

// A maximum, the sum of exp(x - maximum), the first index that has the maximum.
struct Best {
  float top, sum;
  int index;
  __device__ void join(const Best& o) {
    const float t = fmaxf(top, o.top), base = t == -INFINITY ? 0.f : t;
    sum = sum * exp_of(top - base) + o.sum * exp_of(o.top - base);
    if (o.top > top || (o.top == top && static_cast<unsigned>(o.index) < static_cast<unsigned>(index))) index = o.index;
    top = t;
  }
  __device__ void join_warp() {
#pragma unroll
    for (int d = 16; d; d >>= 1) {
      Best o;
      o.top = __shfl_xor_sync(0xffffffffu, top, d);
      o.sum = __shfl_xor_sync(0xffffffffu, sum, d);
      o.index = __shfl_xor_sync(0xffffffffu, index, d);
      // the lower lanes' part first, on both sides of the exchange
      if (threadIdx.x & d) {
        const Best mine = *this;
        *this = o;
        join(mine);
      } else {
        join(o);
      }
    }
  }
};

template <bool BF16>
__device__ __forceinline__ float load1(const void* row, int v) {
  if constexpr (BF16)
    return __uint_as_float(static_cast<uint32_t>(static_cast<const volatile uint16_t*>(row)[v]) << 16);
  else
    return static_cast<const volatile float*>(row)[v];
}

template <bool BF16, int T>
__global__ void __launch_bounds__(T) k_logits(const LogitsParams p) {
  constexpr int W = BF16 ? 8 : 4;    // tokens of a 16-byte vector
  constexpr int kAhead = BF16 ? 2 : 4;
  extern __shared__ uint32_t words[];          // [run + kLead] history, then [run + kLead] biases
  __shared__ Best warps[T / 32];
  __shared__ int again, finish;
  const int tid = threadIdx.x, b = blockIdx.x / p.runs, run = blockIdx.x - b * p.runs;
  const fl_logits_rules& r = p.r;
  const int room = p.run + kLead;
  const bool counts = r.history != nullptr, biases = r.bias_ids != nullptr;
  uint32_t* seen = words;
  int* named = reinterpret_cast<int*>(words + (counts ? room : 0));
  if (counts)
    for (int i = tid; i < room / 4; i += T) reinterpret_cast<uint4*>(seen)[i] = make_uint4(0, 0, 0, 0);
  if (biases)
    for (int i = tid; i < room; i += T) named[i] = std::numeric_limits<int>::max();
  if (tid == 0) again = 0;

  pdl_wait();
  pdl_launch_dependents();
  const uint8_t* row = static_cast<const uint8_t*>(p.x) + static_cast<int64_t>(b) * p.xs * (BF16 ? 2 : 4);
  float* out = p.out ? p.out + static_cast<int64_t>(b) * p.os : nullptr;
  // the row's first token on 16 bytes; without such rows every token goes alone
  const int head = p.vec_x ? min(static_cast<int>((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / (BF16 ? 2 : 4), p.V) : 0;
  const int64_t first = head + static_cast<int64_t>(run) * p.run;      // of the run's vectors
  const int lo = run == 0 ? 0 : static_cast<int>(min(first, static_cast<int64_t>(p.V)));
  const int hi = static_cast<int>(min(first + p.run, static_cast<int64_t>(p.V)));
  const int base = static_cast<int>(min(first, static_cast<int64_t>(p.V))) - kLead;    // token of word 0
  const int nvec = p.vec_x && hi > base + kLead ? (hi - base - kLead) / W : 0;

  // the first vectors are on their way while the history is counted
  uint4 ahead[kAhead];
  auto fetch = [&](int j) {
    if (j >= nvec) return make_uint4(0, 0, 0, 0);
    uint4 f;
    asm volatile("ld.global.cs.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(f.x), "=r"(f.y), "=r"(f.z), "=r"(f.w)
                 : "l"(row + (base + kLead + static_cast<int64_t>(j) * W) * (BF16 ? 2 : 4)));
    return f;
  };
#pragma unroll
  for (int i = 0; i < kAhead; ++i) ahead[i] = fetch(tid + i * T);

  __syncthreads();
  if (counts) {
    const int n = min(max(r.history_lens[b], 0), r.history_max);
    const int prompt = r.prompt_lens ? min(max(r.prompt_lens[b], 0), n) : 0;
    const int32_t* h = r.history + static_cast<int64_t>(b) * r.history_stride;
    auto count = [&](int id, int at) {
      if (id >= lo && id < hi) {
        if (at < prompt)
          atomicOr(seen + (id - base), 0x80000000u);
        else
          atomicAdd(seen + (id - base), 1u);
      }
    };
    int i0 = 0;
    if (p.vec_h) {
#pragma unroll 4
      for (int i = tid; i < n / 4; i += T) {
        const int4 f = __ldg(reinterpret_cast<const int4*>(h) + i);
        count(f.x, 4 * i), count(f.y, 4 * i + 1), count(f.z, 4 * i + 2), count(f.w, 4 * i + 3);
      }
      i0 = n / 4 * 4;
    }
    for (int i = i0 + tid; i < n; i += T) count(__ldg(h + i), i);
  }
  int bias_lo = 0, bias_hi = 0;
  if (biases) {
    bias_lo = min(max(r.bias_offsets[b], 0), r.bias_count);
    bias_hi = min(max(r.bias_offsets[b + 1], bias_lo), r.bias_count);
    for (int i = bias_lo + tid; i < bias_hi; i += T) {
      const int id = __ldg(r.bias_ids + i);
      if (id >= lo && id < hi && atomicMin(named + (id - base), i) != std::numeric_limits<int>::max()) again = 1;
    }
  }
  __syncthreads();

  const float rep = r.repetition ? r.repetition[b] : 1.f, freq = r.frequency ? r.frequency[b] : 0.f;
  const float pres = r.presence ? r.presence[b] : 0.f;
  float inv = 1.f;
  if (r.temperature) {
    const float t = r.temperature[b];
    inv = t > 0.f ? __fdiv_rn(1.f, t) : 1.f;
  }
  const uint32_t* mask = r.allowed ? reinterpret_cast<const uint32_t*>(r.allowed) + static_cast<int64_t>(b) * r.allowed_stride : nullptr;
  const int several = again;
  Best best = {-INFINITY, 0.f, -1};

  auto penalty = [&](float x, uint32_t w) {
    if (r.repetition) x = x > 0.f ? __fdiv_rn(x, rep) : __fmul_rn(x, rep);
    const uint32_t c = w & 0x7fffffffu;
    if (c) {
      if (r.frequency) x = __fsub_rn(x, __fmul_rn(freq, static_cast<float>(c)));
      if (r.presence) x = __fsub_rn(x, pres);
    }
    return x;
  };
  auto biased = [&](float x, int v, int i) {
    x = __fadd_rn(x, __ldg(r.bias + i));
    if (several)
      for (int j = i + 1; j < bias_hi; ++j)
        if (__ldg(r.bias_ids + j) == v) x = __fadd_rn(x, __ldg(r.bias + j));
    return x;
  };
  auto one = [&](int v) {   // a token outside the vectors
    float x = load1<BF16>(row, v);
    if (counts && seen[v - base]) x = penalty(x, seen[v - base]);
    if (biases && named[v - base] != std::numeric_limits<int>::max()) x = biased(x, v, named[v - base]);
    x = __fmul_rn(x, inv);
    if (mask && !(__ldg(mask + (v >> 5)) >> (v & 31) & 1)) x = -INFINITY;
    if (out) out[v] = x;
    best.join(Best{x == x ? x : -INFINITY, x == x ? (x == -INFINITY ? 0.f : 1.f) : x, x > -INFINITY ? v : -1});
  };
  // a run's tokens in ascending order a thread: head, vectors, tail
  if (tid < base + kLead - lo) one(lo + tid);
  auto vector = [&](int j, const uint4& f) {
    const int at = kLead + j * W, v = base + at;
    float x[W];
    if constexpr (BF16) {
#pragma unroll
      for (int e = 0; e < W; ++e) x[e] = __uint_as_float(e & 1 ? (&f.x)[e / 2] & 0xffff0000u : (&f.x)[e / 2] << 16);
    } else {
#pragma unroll
      for (int e = 0; e < W; ++e) x[e] = __uint_as_float((&f.x)[e]);
    }
    if (counts) {
#pragma unroll
      for (int q = 0; q < W / 4; ++q) {
        const uint4 w = reinterpret_cast<const uint4*>(seen + at)[q];
        if (w.x | w.y | w.z | w.w) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if ((&w.x)[e]) x[4 * q + e] = penalty(x[4 * q + e], (&w.x)[e]);
        }
      }
    }
    if (biases) {
#pragma unroll
      for (int e = 0; e < W; ++e)
        if (named[at + e] != std::numeric_limits<int>::max()) x[e] = biased(x[e], v + e, named[at + e]);
    }
#pragma unroll
    for (int e = 0; e < W; ++e) x[e] = __fmul_rn(x[e], inv);
    if (mask) {
      const uint32_t w0 = __ldg(mask + (v >> 5));
      const uint32_t w1 = (v & 31) + W > 32 ? __ldg(mask + (v >> 5) + 1) : 0;
      const uint32_t bits = __funnelshift_r(w0, w1, v & 31);
#pragma unroll
      for (int e = 0; e < W; ++e)
        if (!(bits >> e & 1)) x[e] = -INFINITY;
    }
    if (out) {
      if (p.vec_out) {
#pragma unroll
        for (int q = 0; q < W / 4; ++q)
          __stcs(reinterpret_cast<float4*>(out + v) + q, make_float4(x[4 * q], x[4 * q + 1], x[4 * q + 2], x[4 * q + 3]));
      } else {
#pragma unroll
        for (int e = 0; e < W; ++e) out[v + e] = x[e];
      }
    }
    float top = x[0];
#pragma unroll
    for (int e = 1; e < W; ++e) top = fmaxf(top, x[e]);
    if (top > best.top) {
      best.sum *= exp_of(best.top - top);
      best.top = top;
#pragma unroll
      for (int e = W - 1; e >= 0; --e)
        if (x[e] == top) best.index = v + e;
    }
    const float zero = best.top == -INFINITY ? 0.f : best.top;
    float sum = 0.f;
#pragma unroll
    for (int e = 0; e < W; ++e) sum += exp_of(x[e] - zero);
    best.sum += sum;
  };
  for (int j = tid; j < nvec; j += kAhead * T) {
    uint4 now[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      now[i] = ahead[i];
      ahead[i] = fetch(j + (kAhead + i) * T);
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (j + i * T < nvec) vector(j + i * T, now[i]);
  }
  for (int v = base + kLead + nvec * W + tid; v < hi; v += T) one(v);

  best.join_warp();
  if ((tid & 31) == 0) warps[tid >> 5] = best;
  __syncthreads();
  auto write = [&](const Best& all) {
    const float log_sum = logf(all.sum);
    const bool none = all.top == -INFINITY;
    p.token[b] = all.index;
    if (p.lse) p.lse[b] = all.sum == 0.f ? -INFINITY : (none ? 0.f : all.top) + log_sum;
    if (p.logprob) p.logprob[b] = all.sum == 0.f ? -INFINITY : -log_sum;
  };
  if (tid < 32) {
    best = tid < T / 32 ? warps[tid] : Best{-INFINITY, 0.f, -1};
    best.join_warp();
    if (tid == 0) {
      finish = 0;
      if (p.runs == 1) {
        write(best);
      } else {
        __stcg(reinterpret_cast<float4*>(p.part + static_cast<int64_t>(b) * p.runs + run),
               make_float4(best.top, best.sum, __int_as_float(best.index), 0.f));
        finish = atom_add_acq_rel_gpu(p.cnt + b, 1) == p.runs - 1;
        if (finish) p.cnt[b] = 0;
      }
    }
  }
  __syncthreads();
  if (!finish) return;
  best = {-INFINITY, 0.f, -1};
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
    if (tid == 0) write(best);
  }
}

bool aligned(const void* p, int n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// Tokens of a run: the longest that still gives every SM eight of them, so that
// the history is read by few; short runs where rows are few.
int run_length(int B, int V) {
  const long long want = 8ll * flh::sm_count();
  int run = kRunMax;
  while (run > kRunMin && (V + run - 1ll) / run * B < want) run /= 2;
  return run;
}
int run_count(int V, int run) { return static_cast<int>((V + run - 1ll) / run); }

template <bool BF16, int T>
int launch(const LogitsParams& p, int B, size_t smem, cudaStream_t s) {
  static bool ready[64] = {false};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 0 && dev < 64 && !ready[dev]) {
    if (cudaFuncSetAttribute(k_logits<BF16, T>, cudaFuncAttributeMaxDynamicSharedMemorySize, 2 * (kRunMax + kLead) * 4) != cudaSuccess) {
      cudaGetLastError();
      return FL_ERR_CUDA;
    }
    ready[dev] = true;
  }
  return flh::launch_early(k_logits<BF16, T>, dim3(static_cast<unsigned>(B) * p.runs), dim3(T), smem, s, p);
}

bool logits_args(int B, int V) { return B >= 1 && V >= 1 && V < (1 << 30) && B <= (1 << 30); }

}  // namespace

extern "C" int fl_logits_process_workspace(int B, int V, size_t* out) {
  if (!out || !logits_args(B, V)) return FL_ERR_ARG;
  const int rows = B < kRowsMax ? B : kRowsMax;
  *out = kScratchOff + static_cast<size_t>(rows) * run_count(V, run_length(B, V)) * sizeof(Partial);
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
  if (out == logits && out && (bf16 || out_stride != logits_stride)) return FL_ERR_ARG;
  if (!r.history != !r.history_lens || (r.history && (r.history_max < 0 || r.history_max >= 1 << 30 || r.history_stride < r.history_max)))
    return FL_ERR_ARG;
  if (!r.history && (r.prompt_lens || r.repetition || r.frequency || r.presence)) return FL_ERR_ARG;
  if (!r.bias_offsets != !r.bias_ids || !r.bias_ids != !r.bias || (r.bias && r.bias_count < 0)) return FL_ERR_ARG;
  if (r.allowed && r.allowed_stride < (V + 31) / 32) return FL_ERR_ARG;
  size_t need = 0;
  fl_logits_process_workspace(B, V, &need);
  if (ws_bytes < need) return FL_ERR_WORKSPACE;

  LogitsParams p = {};
  p.xs = logits_stride, p.os = out_stride, p.r = r, p.V = V;
  p.run = run_length(B, V);
  // a long history is worth longer runs: each of a row's CTAs reads it
  while (r.history && p.run < kRunMax && p.run < r.history_max / 8) p.run *= 2;
  p.runs = run_count(V, p.run);
  p.part = reinterpret_cast<Partial*>(static_cast<uint8_t*>(ws) + kScratchOff);
  p.cnt = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(ws) + kTicketOff);
  p.vec_x = 1;
  p.vec_h = aligned(r.history, 16) && r.history_stride % 4 == 0;
  // a row's tokens on 16 bytes are so in both (rows shift both alike)
  const int64_t size = bf16 ? 2 : 4;
  const uintptr_t in0 = reinterpret_cast<uintptr_t>(logits) / size, out0 = reinterpret_cast<uintptr_t>(out) / 4;
  p.vec_out = out && (in0 - out0) % 4 == 0 && (logits_stride - out_stride) % 4 == 0;
  const size_t smem = static_cast<size_t>(p.run + kLead) * 4 * ((r.history ? 1 : 0) + (r.bias ? 1 : 0));
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  for (int b = 0; b < B;) {
    int n = B - b < kRowsMax ? B - b : kRowsMax;
    const long long most = 0x7fffffffll / p.runs;
    if (n > most) n = static_cast<int>(most);
    LogitsParams q = p;
    q.x = static_cast<const uint8_t*>(logits) + static_cast<int64_t>(b) * logits_stride * size;
    q.out = out ? out + static_cast<int64_t>(b) * out_stride : nullptr;
    q.token = token + b, q.lse = lse ? lse + b : nullptr, q.logprob = logprob ? logprob + b : nullptr;
    auto row = [&](auto*& list, int64_t stride) { if (list) list += b * stride; };
    row(q.r.history, r.history_stride), row(q.r.history_lens, 1), row(q.r.prompt_lens, 1), row(q.r.repetition, 1);
    row(q.r.frequency, 1), row(q.r.presence, 1), row(q.r.bias_offsets, 1), row(q.r.allowed, r.allowed_stride), row(q.r.temperature, 1);
    const int rc = p.run > 2048 ? (bf16 ? launch<true, 512>(q, n, smem, s) : launch<false, 512>(q, n, smem, s))
                                : (bf16 ? launch<true, 256>(q, n, smem, s) : launch<false, 256>(q, n, smem, s));
    if (rc != FL_OK) return rc;
    b += n;
  }
  return FL_OK;
}
