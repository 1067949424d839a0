// The write of new keys and values into the 8-bit paged cache.
//
// A CTA owns one (block of a sequence, kv head, keys or values): nobody else
// writes that block's codes or scale.  It reads the block's new tokens once
// (16 bytes a thread and load, kept in registers), takes the largest
// magnitude, and so the scale: the least 2^e with max / 2^e <= 448 or 127.
// If the block holds earlier tokens whose scale was larger it keeps that one;
// if it was smaller, their codes are moved to the new scale.  Then the new
// codes are written.  Division by a power of two is exact, so a code is one
// rounding of its bf16 input.  Bound by HBM: 3 bytes an element.  The kernel is
// built for each block size, so that a thread keeps no more registers than it
// has vectors and more CTAs fit an SM.  Measured: 12.5K tokens of prompts, 8 heads
// of 128 (95 MB) 26 us from cold caches, and 17.5 us in a chain of calls, 5.4 TB/s.
// The thread that finds the CTA's sequence hands on what it has read of it (read
// once more by all: 48 single tokens 4.2 us, not 4.0).
#include "fl_kv8.cuh"

using namespace flkv;

namespace {

struct Half {   // keys, or values
  const __nv_bfloat16* src;
  int64_t stride;
  uint8_t* dst;
  float* scale;
};
struct AppendParams {
  Half k, v;
  Seqs seqs;
  int num_blocks, heads;
  int32_t* status;
};

// Four values to four codes.  Integers: adding 1.5 * 2^23 leaves the nearest
// even integer in the sum's low bits.
template <int FMT>
__device__ __forceinline__ uint32_t quant4(float a, float b, float c, float d) {
  if constexpr (FMT == FL_KV8_E4M3) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | hi << 16;
  } else {
    constexpr float kMagic = 12582912.f;
    const uint32_t ab = __byte_perm(__float_as_uint(a + kMagic), __float_as_uint(b + kMagic), 0x0040);
    const uint32_t cd = __byte_perm(__float_as_uint(c + kMagic), __float_as_uint(d + kMagic), 0x0040);
    return __byte_perm(ab, cd, 0x5410);
  }
}
// Eight bf16 values to codes by a scale that is not a power of two.
template <int FMT>
__device__ __noinline__ uint2 divided8(uint4 x, float scale) {
  constexpr float kTop = FMT == FL_KV8_E4M3 ? 448.f : 127.f;
  const uint32_t a[4] = {x.x, x.y, x.z, x.w};
  uint32_t out[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float f[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const uint32_t w = a[2 * i + t / 2];
      f[t] = fminf(fmaxf(__uint_as_float(t & 1 ? w & 0xffff0000u : w << 16) / scale, -kTop), kTop);
    }
    out[i] = quant4<FMT>(f[0], f[1], f[2], f[3]);
  }
  return make_uint2(out[0], out[1]);
}
template <int FMT>
__device__ __forceinline__ float code_value(uint32_t c) {
  if constexpr (FMT == FL_KV8_E4M3) {
    const __half_raw h = __nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(c & 0xffu), __NV_E4M3);
    return __half2float(*reinterpret_cast<const __half*>(&h));
  }
  return static_cast<float>(static_cast<int8_t>(c));
}

// A CTA's work: slots [lo, hi) of page `page` of sequence b, from the call's
// token `row` on.  b is -1 without work.
struct Block {
  int b, page, lo, hi, row;
};
__device__ __forceinline__ Block block_of(const SeqInfo& q, int block, int b, int j) {
  const PageRun run = written_pages(q, block);
  const int page = run.first + j, lo = max(max(q.kv - q.n, 0) - page * block, 0);   // (from the first position written)
  return {j < run.n ? b : -1, page, lo, min(q.kv - page * block, block), q.start + (page * block + lo - (q.kv - q.n))};
}
// The x-th written block of the batch.
template <int THREADS>
__device__ __forceinline__ Block find_block(const Seqs& s, int block, int x) {
  if (s.B == 1) return block_of(seq_info(s, 0, block), block, 0, x);
  __shared__ int scan[THREADS / 32];
  __shared__ Block hit;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) hit.b = -1;
  int base = 0;
  for (int c = 0; c < s.B && x >= base; c += THREADS) {
    SeqInfo q = {0, 0, 0, false};
    if (c + tid < s.B) q = seq_info(s, c + tid, block);
    const int n = written_pages(q, block).n;
    int inc = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += u;
    }
    __syncthreads();
    if (lane == 31) scan[warp] = inc;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
      if (w < warp) before += scan[w];
      all += scan[w];
    }
    const int mine = base + before + inc - n;
    if (x >= mine && x < mine + n) hit = block_of(q, block, c + tid, x - mine);
    base += all;
  }
  __syncthreads();
  return hit;
}

template <int FMT, int D, int BLK>
struct ApCfg {
  static constexpr int kAll = BLK * D / 8;                    // vectors of 8 elements of a block
  static constexpr int kThreads = kAll < 256 ? kAll : 256;
  static constexpr int kVecs = kAll / kThreads;               // of a thread, at most
};

template <int FMT, int D, int BLK>
__global__ void __launch_bounds__(ApCfg<FMT, D, BLK>::kThreads) k_kv8_append(const AppendParams p) {
  using C = ApCfg<FMT, D, BLK>;
  constexpr int kThreads = C::kThreads, kVecs = C::kVecs, kWarps = kThreads / 32;
  __shared__ float s_red[kWarps];
  pdl_launch_dependents();
  pdl_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int b, j;
  if (blockIdx.x == gridDim.x - 1) {   // past the last block: records the sequences that are left out
    if (blockIdx.y == 0 && blockIdx.z == 0)
      for (int i = tid; i < p.seqs.B; i += kThreads)
        if (seq_info(p.seqs, i, BLK).bad) set_status(p.status, FL_ERR_DEVICE_CHECK, 53);
    return;
  }
  const Block at = find_block<kThreads>(p.seqs, BLK, blockIdx.x);
  if (at.b < 0) return;
  const int lo = at.lo, hi = at.hi;
  const int head = blockIdx.y;
  const bool vals = blockIdx.z != 0;
  const Half h = {vals ? p.v.src : p.k.src, vals ? p.v.stride : p.k.stride, vals ? p.v.dst : p.k.dst,
                  vals ? p.v.scale : p.k.scale};
  const int page = page_block(p.seqs, at.b, at.page, p.num_blocks);
  const __nv_bfloat16* src = h.src + at.row * h.stride + head * D;
  const int nv = (hi - lo) * (D / 8);
  uint4 x[kVecs];
  uint32_t top2 = 0;   // the largest magnitudes' bits, of either half of a word
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int v = i * kThreads + tid;
    x[i] = make_uint4(0, 0, 0, 0);
    if (v < nv) x[i] = __ldcs(reinterpret_cast<const uint4*>(src + static_cast<int64_t>(v / (D / 8)) * h.stride + v % (D / 8) * 8));
  }
  if (page < 0) {
    if (tid == 0) set_status(p.status, FL_ERR_DEVICE_CHECK, 50);
    return;
  }
  const int64_t tile = static_cast<int64_t>(page) * p.heads + head;
  uint8_t* codes = h.dst + tile * BLK * D;
  const float old = lo > 0 ? h.scale[tile] : 0.f;
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    top2 = __vmaxu2(top2, __vmaxu2(x[i].x & 0x7fff7fffu, x[i].y & 0x7fff7fffu));
    top2 = __vmaxu2(top2, __vmaxu2(x[i].z & 0x7fff7fffu, x[i].w & 0x7fff7fffu));
  }
  uint32_t top = max(top2 & 0xffffu, top2 >> 16);
  if (top >= 0x7f80u) {
    // infinities become the largest finite bf16, NaN 0
    set_status(p.status, FL_ERR_RANGE, 51);
    top = 0;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      auto mend = [&](uint32_t a) {
#pragma unroll
        for (int h = 0; h < 32; h += 16) {
          const uint32_t e = (a >> h) & 0x7fffu;
          if (e >= 0x7f80u) a = (a & ~(0xffffu << h)) | (e == 0x7f80u ? ((a >> h) & 0x8000u) | 0x7f7fu : 0u) << h;
          top = max(top, (a >> h) & 0x7fffu);
        }
        return a;
      };
      x[i] = make_uint4(mend(x[i].x), mend(x[i].y), mend(x[i].z), mend(x[i].w));
    }
  }
  top = __reduce_max_sync(0xffffffffu, top);
  if (lane == 0) s_red[warp] = __uint_as_float(top);
  __syncthreads();   // (also: every thread has read the old scale)
#pragma unroll
  for (int w = 0; w < kWarps; ++w) top = max(top, __float_as_uint(s_red[w]));
  // top = m 2^e with 1 <= m < 2; the range's end is 1.75 * 2^8 or 1.984375 * 2^6
  int e = static_cast<int>(top >> 7) - 127 - (FMT == FL_KV8_E4M3 ? 8 : 6);
  if ((top & 0x7fu) > (FMT == FL_KV8_E4M3 ? 0x60u : 0x7eu)) ++e;
  const float need = pow2i(max(e, -126));
  const bool keep = lo > 0 && old >= need;
  const float scale = keep ? old : need;
  if (lo > 0 && !keep) {
    // earlier tokens move to the larger scale, rounded once more
    const float ratio = old / scale;
    for (int v = tid; v < lo * (D / 16); v += kThreads) {
      const uint4 c = reinterpret_cast<const uint4*>(codes)[v];
      auto move = [&](uint32_t a) {
        return quant4<FMT>(code_value<FMT>(a) * ratio, code_value<FMT>(a >> 8) * ratio, code_value<FMT>(a >> 16) * ratio,
                           code_value<FMT>(a >> 24) * ratio);
      };
      reinterpret_cast<uint4*>(codes)[v] = make_uint4(move(c.x), move(c.y), move(c.z), move(c.w));
    }
  }
  // 1 / scale: exact for a power of two; a scale that a caller chose is divided by,
  // out of the way of the common loop (12.5K tokens of prompts as int8: 18.8 us with
  // the divisions in it, 17.3 without)
  const bool pow2 = (__float_as_uint(scale) & 0x7fffffu) == 0;
  const float inv = 1.f / scale;
  uint2* dst = reinterpret_cast<uint2*>(codes + static_cast<int64_t>(lo) * D);
  if (pow2) {   // (of the largest value's own making, or larger: nothing is outside the range)
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int v = i * kThreads + tid;
      const uint32_t a[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
      float f[8];
#pragma unroll
      for (int t = 0; t < 4; ++t) f[2 * t] = __uint_as_float(a[t] << 16) * inv, f[2 * t + 1] = __uint_as_float(a[t] & 0xffff0000u) * inv;
      if (v < nv) dst[v] = make_uint2(quant4<FMT>(f[0], f[1], f[2], f[3]), quant4<FMT>(f[4], f[5], f[6], f[7]));
    }
  } else {
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
      if (i * kThreads + tid < nv) dst[i * kThreads + tid] = divided8<FMT>(x[i], scale);
  }
  if (tid == 0) h.scale[tile] = scale;
}

template <int FMT, int D>
int launch_append(const AppendParams& p, int block, dim3 grid, cudaStream_t s) {
  switch (block) {
    case 16: return flh::launch_early(k_kv8_append<FMT, D, 16>, grid, ApCfg<FMT, D, 16>::kThreads, 0, s, p);
    case 32: return flh::launch_early(k_kv8_append<FMT, D, 32>, grid, ApCfg<FMT, D, 32>::kThreads, 0, s, p);
    case 64: return flh::launch_early(k_kv8_append<FMT, D, 64>, grid, ApCfg<FMT, D, 64>::kThreads, 0, s, p);
    default: return flh::launch_early(k_kv8_append<FMT, D, 128>, grid, ApCfg<FMT, D, 128>::kThreads, 0, s, p);
  }
}

}  // namespace

extern "C" int fl_kv8_append(const void* k, int64_t k_stride, const void* v, int64_t v_stride, const fl_kv8_cache* cache,
                             const fl_kv8_seqs* seqs, void* status, fl_stream_t stream) {
  if (!k || !v || !status || !flh::aligned16(k) || !flh::aligned16(v) || !flh::aligned16(status)) return FL_ERR_ARG;
  const int rc = flh::kv8_check(cache, seqs);
  if (rc != FL_OK) return rc;
  const int64_t width = static_cast<int64_t>(cache->kv_heads) * cache->head_dim;
  if (k_stride < width || v_stride < width || k_stride % 8 || v_stride % 8) return FL_ERR_ARG;
  if (cache->kv_heads > 65535) return FL_ERR_UNSUPPORTED;
  AppendParams p;
  p.k = {static_cast<const __nv_bfloat16*>(k), k_stride, static_cast<uint8_t*>(cache->k), cache->k_scale};
  p.v = {static_cast<const __nv_bfloat16*>(v), v_stride, static_cast<uint8_t*>(cache->v), cache->v_scale};
  p.seqs = flh::seqs_of(*seqs);
  p.num_blocks = cache->num_blocks, p.heads = cache->kv_heads;
  p.status = static_cast<int32_t*>(status);
  // n new tokens touch at most (n - 1) / block + 2 blocks, and never more than
  // n; so the batch at most the sum of either over its sequences
  long long most = seqs->T / cache->block + 2ll * seqs->B;
  if (most > seqs->T) most = seqs->T;
  if (most > 0x7ffffffell) return FL_ERR_UNSUPPORTED;
  const dim3 grid(static_cast<unsigned>(most) + 1, cache->kv_heads, 2);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (cache->format == FL_KV8_E4M3)
    return cache->head_dim == 64 ? launch_append<FL_KV8_E4M3, 64>(p, cache->block, grid, s)
                                 : launch_append<FL_KV8_E4M3, 128>(p, cache->block, grid, s);
  return cache->head_dim == 64 ? launch_append<FL_KV8_INT8, 64>(p, cache->block, grid, s)
                               : launch_append<FL_KV8_INT8, 128>(p, cache->block, grid, s);
}

extern "C" int fl_kv8_test_pages(const fl_kv8_seqs* seqs, int num_blocks, int block, int window, int b, long long* out) {
  if (!seqs || !out || !seqs->kv_lens || !seqs->block_table || num_blocks < 1 || block < 1 || window < 0 || b < 0 ||
      b >= seqs->B || seqs->T > (1 << 29) || seqs->max_blocks > (1 << 30) / block)
    return FL_ERR_ARG;
  if (window >= seqs->max_blocks * block) window = 0;
  const Seqs s = flh::seqs_of(*seqs);
  const SeqInfo q = seq_info(s, b, block);
  const PageRun runs[2] = {written_pages(q, block), read_pages(q, block, window)};
  out[0] = q.start, out[1] = q.n, out[2] = q.kv;
  for (int i = 0; i < 2; ++i) {
    out[3 + 3 * i] = runs[i].first, out[4 + 3 * i] = runs[i].n, out[5 + 3 * i] = 0;
    for (int pg = 0; pg < runs[i].n; ++pg) out[5 + 3 * i] += page_block(s, b, runs[i].first + pg, num_blocks) < 0;
  }
  return FL_OK;
}
