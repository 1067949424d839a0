// Shared pieces of the 8-bit key/value cache: its sequences, its codes.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "fl_common.cuh"

namespace flkv {

using namespace fl;

// Device view of fl_kv8_seqs.  The lists are read with every bound checked,
// so that no content of theirs can lead outside the arrays.
struct Seqs {
  const int32_t* cu_q;
  const int32_t* kv_lens;
  const int32_t* table;
  int T, B, max_q, max_blocks;
};

// Query rows [start, start + n) of sequence b and its cache length.  bad: the
// lists name rows or tokens that the arrays have not; the sequence is left out
// (cut to the arrays, its rows would stand at other positions than their own).
struct SeqInfo {
  int start, n, kv;
  bool bad;
};
__host__ __device__ __forceinline__ SeqInfo seq_info(const Seqs& s, int b, int block) {
  SeqInfo r;
  int end;
  if (s.cu_q) {
    r.start = s.cu_q[b], end = s.cu_q[b + 1];
  } else {
    r.start = b * (s.T / s.B), end = r.start + s.T / s.B;
  }
  r.kv = max(s.kv_lens[b], 0);
  r.bad = r.start < 0 || end < r.start || end > s.T || end - r.start > s.max_q ||
          (end > r.start && r.kv > s.max_blocks * block);
  r.n = r.bad ? 0 : end - r.start;
  if (r.n == 0) r.start = r.kv = 0;
  return r;
}

// The cache block of page pg of sequence b, or -1 where the table has no entry
// or names a block that the cache has not.
__host__ __device__ __forceinline__ int page_block(const Seqs& s, int b, int pg, int num_blocks) {
  if (pg < 0 || pg >= s.max_blocks) return -1;
  const int id = s.table[static_cast<int64_t>(b) * s.max_blocks + pg];
  return id >= 0 && id < num_blocks ? id : -1;
}

// Pages [first, first + n) of a sequence that its new tokens are written to.
struct PageRun {
  int first, n;
};
__host__ __device__ __forceinline__ PageRun written_pages(const SeqInfo& q, int block) {
  const int p0 = max(q.kv - q.n, 0);
  return q.kv > p0 ? PageRun{p0 / block, (q.kv - 1) / block - p0 / block + 1} : PageRun{0, 0};
}
// The first token that any row sees, and the pages with a token that one sees.
__host__ __device__ __forceinline__ int first_seen(const SeqInfo& q, int window) {
  return window ? max(0, q.kv - q.n + 1 - window) : 0;
}
__host__ __device__ __forceinline__ PageRun read_pages(const SeqInfo& q, int block, int window) {
  const int first = first_seen(q, window) / block;
  return PageRun{first, (q.kv + block - 1) / block - first};
}

// ------------------------------------------------------------------ codes
// Two 8-bit codes (the low 16 bits, or with HI the high 16) as an f16 pair.
// Both formats are exact in f16.
template <int FMT, bool HI>
__device__ __forceinline__ uint32_t code_pair_f16(uint32_t w) {
  if constexpr (FMT == FL_KV8_E4M3) {
    uint32_t d;
    const uint16_t h = static_cast<uint16_t>(HI ? w >> 16 : w);
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"(h));
    return d;
  } else {
    // w holds code + 128 in every byte: f16 1024 + u has u in its last byte
    const uint32_t u = __byte_perm(w, 0x64646464u, HI ? 0x4342u : 0x4140u);
    const __half2 v = __hsub2(*reinterpret_cast<const __half2*>(&u), __half2half2(__ushort_as_half(0x6480)));  // 1152
    return *reinterpret_cast<const uint32_t*>(&v);
  }
}
// What code_pair_f16 wants: the raw codes, or for integers code + 128.
template <int FMT>
__device__ __forceinline__ uint32_t bias_codes(uint32_t w) {
  return FMT == FL_KV8_E4M3 ? w : w ^ 0x80808080u;
}

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Arguments of the attention kernels.  A launch serves the sequences whose
// rows (query heads of a kv head x tokens) number in (rows_lo, rows_hi].
struct AttnParams {
  const __nv_bfloat16* q;
  __nv_bfloat16* out;
  float* lse;
  const float* ks;
  const float* vs;
  float* part;
  int32_t* cnt;
  int32_t* status;
  int64_t qs, os;
  Seqs seqs;
  int num_blocks, block, heads, group, Hq, window;
  int rows_lo, rows_hi;
  float scale2;   // scale * log2(e)
};

constexpr float kLn2 = 0.69314718055994530942f;

// Runs of units: all units of the batch lie in one line, sequence by
// sequence, and CTA c of P takes [c U / P, (c + 1) U / P).
__host__ __device__ __forceinline__ long long unit_begin(int c, long long U, int P) { return c * U / P; }
__host__ __device__ __forceinline__ int cta_of_unit(long long u, long long U, int P) {
  return static_cast<int>(((u + 1) * P - 1) / U);
}

// U, P and the sequence that the first unit of CTA c of P lies in (b, and the
// units before it), by a scan over the sequences.  All THREADS threads take
// part.  P is at most `ctas` and ceil(U / least), 0 without units.
struct Start {
  long long U, base;
  int P, b;
};
// scratch: shared memory for THREADS / 32 + 2 numbers, free again after a barrier.
template <int THREADS, typename F>
__device__ __forceinline__ Start find_start(long long* scratch, int B, int c0, int ctas, int least, F&& units_of) {
  long long* scan = scratch;
  long long* hit = scratch + THREADS / 32;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const bool one = B <= THREADS;   // with one chunk of sequences the first pass has it all
  long long U = 0;
  auto parts = [&](long long n) { return static_cast<int>(min(static_cast<long long>(ctas), (n + least - 1) / least)); };
  for (int pass = 0; pass < 2; ++pass) {
    long long base = 0;
    for (int c = 0; c < B; c += THREADS) {
      const long long n = c + tid < B ? units_of(c + tid) : 0;
      long long inc = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += v;
      }
      __syncthreads();
      if (lane == 31) scan[warp] = inc;
      __syncthreads();
      long long before = 0, all = 0;
#pragma unroll
      for (int w = 0; w < THREADS / 32; ++w) {
        if (w < warp) before += scan[w];
        all += scan[w];
      }
      if (one) U = all;
      if (one || pass == 1) {
        const int P = parts(U);
        const long long u0 = c0 < P ? unit_begin(c0, U, P) : U;
        const long long mine = base + before + inc - n;
        if (u0 >= mine && u0 < mine + n) {
          hit[0] = c + tid;
          hit[1] = mine;
        }
      }
      base += all;
    }
    U = base;
    if (one) break;
  }
  __syncthreads();
  return {U, hit[1], parts(U), static_cast<int>(hit[0])};
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ void mbar_expect_tx(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}

// The 16-byte chunk c of row r of a swizzled tile of D-byte rows (128-byte
// rows: c ^ r % 8; 64-byte rows: c ^ (r / 2) % 4).
template <int D>
__device__ __forceinline__ int chunk_at(int r, int c) {
  return r * D + ((D == 128 ? c ^ (r & 7) : c ^ ((r >> 1) & 3)) << 4);
}

// A query row's power of two: e with its largest magnitude in [2^e, 2^(e+1)),
// from the largest bf16 magnitude bits.
__device__ __forceinline__ int row_exponent(uint32_t top) {
  return top ? min(max(static_cast<int>(top >> 7) - 127, -126), 126) : 0;
}

// 2^e for -126 <= e <= 127
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }

}  // namespace flkv

namespace flh {

// The device's view of the sequences.  max_q is a bound that may be loose; no
// sequence has more than T rows.
inline flkv::Seqs seqs_of(const fl_kv8_seqs& s) {
  return {s.cu_q, s.kv_lens, s.block_table, s.T, s.B, s.max_q < s.T ? s.max_q : s.T, s.max_blocks};
}

// Arguments that fl_kv8_append and fl_kv8_attention share.
inline int kv8_check(const fl_kv8_cache* c, const fl_kv8_seqs* s) {
  if (!c || !s || !c->k || !c->v || !c->k_scale || !c->v_scale || !s->kv_lens || !s->block_table) return FL_ERR_ARG;
  if (!aligned16(c->k) || !aligned16(c->v) || (reinterpret_cast<uintptr_t>(c->k_scale) & 3u) ||
      (reinterpret_cast<uintptr_t>(c->v_scale) & 3u) || (reinterpret_cast<uintptr_t>(s->cu_q) & 3u) ||
      (reinterpret_cast<uintptr_t>(s->kv_lens) & 3u) || (reinterpret_cast<uintptr_t>(s->block_table) & 3u))
    return FL_ERR_ARG;
  if (c->num_blocks < 1 || c->kv_heads < 1 || s->T < 1 || s->B < 1 || s->max_q < 1 || s->max_blocks < 1) return FL_ERR_ARG;
  if (c->format != FL_KV8_E4M3 && c->format != FL_KV8_INT8) return FL_ERR_ARG;
  if (!s->cu_q && (s->T % s->B || s->T / s->B > s->max_q)) return FL_ERR_ARG;
  if ((c->block != 16 && c->block != 32 && c->block != 64 && c->block != 128) ||
      (c->head_dim != 64 && c->head_dim != 128))
    return FL_ERR_UNSUPPORTED;
  if (static_cast<long long>(c->num_blocks) * c->kv_heads > 0x7fffffffll / c->block) return FL_ERR_UNSUPPORTED;
  // positions, and their differences with a window, fit 32 bits
  if (s->T > (1 << 29) || s->max_blocks > (1 << 30) / c->block) return FL_ERR_UNSUPPORTED;
  return FL_OK;
}

}  // namespace flh
