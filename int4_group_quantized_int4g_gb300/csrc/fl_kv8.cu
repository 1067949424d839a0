// The write of new keys and values into the 8-bit paged cache.
//
// A CTA owns one (block of a sequence, kv head, keys or values): nobody else
// writes that block's codes or scale.  It reads the block's new tokens once
// (16 bytes a thread and load, kept in registers), takes the largest
// magnitude, and so the scale: the least 2^e with max / 2^e <= 448 or 127.
// If the block holds earlier tokens whose scale was larger it keeps that one;
// if it was smaller, their codes are moved to the new scale.  Then the new
// codes are written.  Division by a power of two is exact, so a code is one
// rounding of its bf16 input.  Bound by HBM: 3 bytes an element.
#include "fl_kv8.cuh"

using namespace flkv;

namespace {

constexpr int kApThreads = 256;

struct AppendParams {
  const __nv_bfloat16* src[2];
  int64_t stride[2];
  uint8_t* dst[2];
  float* scale[2];
  Seqs seqs;
  int num_blocks, block, heads;
  int32_t* status;
};

__device__ __forceinline__ uint32_t quant_byte(float x, int fmt) {
  if (fmt == FL_KV8_E4M3) return __nv_cvt_float_to_fp8(x, __NV_SATFINITE, __NV_E4M3);
  return static_cast<uint32_t>(static_cast<int>(rintf(x))) & 0xffu;
}
__device__ __forceinline__ float code_value(uint32_t c, int fmt) {
  if (fmt == FL_KV8_E4M3) {
    const __half_raw h = __nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(c), __NV_E4M3);
    return __half2float(*reinterpret_cast<const __half*>(&h));
  }
  return static_cast<float>(static_cast<int8_t>(c));
}

template <int FMT, int D>
__global__ void __launch_bounds__(kApThreads) k_kv8_append(const AppendParams p) {
  constexpr int kVecs = 128 * D / 8 / kApThreads;   // vectors of 8 elements a thread, at most
  __shared__ int s_scan[kApThreads / 32];
  __shared__ int s_hit[2];
  __shared__ float s_red[kApThreads / 32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // the CTA's sequence and block: the blockIdx.x-th touched block of the batch
  int b = 0, j = blockIdx.x;
  if (p.seqs.B > 1) {
    if (tid == 0) s_hit[0] = -1;
    int base = 0;
    bool found = false;
    for (int c = 0; c < p.seqs.B && !found; c += kApThreads) {
      const int n = c + tid < p.seqs.B ? written_pages(seq_info(p.seqs, c + tid, p.block), p.block).n : 0;
      int inc = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += u;
      }
      __syncthreads();
      if (lane == 31) s_scan[warp] = inc;
      __syncthreads();
      int before = 0, all = 0;
#pragma unroll
      for (int w = 0; w < kApThreads / 32; ++w) {
        if (w < warp) before += s_scan[w];
        all += s_scan[w];
      }
      const int mine = base + before + inc - n;
      if (static_cast<int>(blockIdx.x) >= mine && static_cast<int>(blockIdx.x) < mine + n) {
        s_hit[0] = c + tid;
        s_hit[1] = blockIdx.x - mine;
      }
      base += all;
      found = static_cast<int>(blockIdx.x) < base;
    }
    __syncthreads();
    b = s_hit[0];
    j = s_hit[1];
    if (b < 0) return;
  }
  const SeqInfo q = seq_info(p.seqs, b, p.block);
  const PageRun run = written_pages(q, p.block);
  if (j >= run.n) return;
  const int p0 = max(q.kv - q.n, 0);           // first position written
  const int jb = run.first + j;
  const int lo = max(p0 - jb * p.block, 0);    // slots [lo, hi) of the block are written
  const int hi = min(q.kv - jb * p.block, p.block);
  const int head = blockIdx.y, kv = blockIdx.z;
  const int page = page_block(p.seqs, b, jb, p.num_blocks);
  if (page < 0) {
    if (tid == 0) set_status(p.status, FL_ERR_DEVICE_CHECK, 50);
    return;
  }
  const int64_t tile = static_cast<int64_t>(page) * p.heads + head;
  uint8_t* codes = p.dst[kv] + tile * p.block * D;
  // row of the first written token in the call's tokens
  const int64_t row0 = static_cast<int64_t>(q.start) + (jb * p.block + lo - (q.kv - q.n));
  const __nv_bfloat16* src = p.src[kv] + row0 * p.stride[kv] + head * D;
  const int nv = (hi - lo) * (D / 8);
  uint4 x[kVecs];
  float top = 0.f;
  bool odd = false;   // an infinity or NaN
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int v = i * kApThreads + tid;
    x[i] = make_uint4(0, 0, 0, 0);
    if (v < nv) x[i] = *reinterpret_cast<const uint4*>(src + static_cast<int64_t>(v / (D / 8)) * p.stride[kv] + v % (D / 8) * 8);
  }
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    uint32_t* a = &x[i].x;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      // an infinity becomes the largest finite bf16, a NaN 0
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t e = (a[t] >> (16 * h)) & 0x7fffu;
        if (e >= 0x7f80u) {
          odd = true;
          const uint32_t keep = e == 0x7f80u ? ((a[t] >> (16 * h)) & 0x8000u) | 0x7f7fu : 0u;
          a[t] = (a[t] & ~(0xffffu << (16 * h))) | (keep << (16 * h));
        }
      }
      top = fmaxf(top, fmaxf(fabsf(__uint_as_float(a[t] << 16)), fabsf(__uint_as_float(a[t] & 0xffff0000u))));
    }
  }
  if (odd) set_status(p.status, FL_ERR_RANGE, 51);
  const float old = lo > 0 ? p.scale[kv][tile] : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (lane == 0) s_red[warp] = top;
  __syncthreads();   // (also: every thread has read the old scale)
#pragma unroll
  for (int w = 0; w < kApThreads / 32; ++w) top = fmaxf(top, s_red[w]);
  // top = m 2^e with 1 <= m < 2; the range's end is 1.75 * 2^8 or 1.984375 * 2^6
  const uint32_t bits = __float_as_uint(top);
  int e = static_cast<int>(bits >> 23) - 127 - (FMT == FL_KV8_E4M3 ? 8 : 6);
  if ((bits & 0x7fffffu) > (FMT == FL_KV8_E4M3 ? 0x600000u : 0x7e0000u)) ++e;
  const float need = pow2i(max(e, -126));
  const bool keep = lo > 0 && old >= need;
  const float scale = keep ? old : need;
  if (lo > 0 && !keep) {
    // earlier tokens move to the larger scale, rounded once more
    const float ratio = old / scale;
    for (int v = tid; v < lo * (D / 16); v += kApThreads) {
      uint4 c = reinterpret_cast<const uint4*>(codes)[v];
      uint32_t* a = &c.x;
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        uint32_t o = 0;
#pragma unroll
        for (int h = 0; h < 4; ++h) o |= quant_byte(code_value((a[t] >> (8 * h)) & 0xffu, FMT) * ratio, FMT) << (8 * h);
        a[t] = o;
      }
      reinterpret_cast<uint4*>(codes)[v] = c;
    }
  }
  // 1 / scale: exact for a power of two; a scale that a caller chose is divided by
  const bool pow2 = (__float_as_uint(scale) & 0x7fffffu) == 0;
  const float inv = 1.f / scale;
  const float most = FMT == FL_KV8_E4M3 ? 448.f : 127.f;
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int v = i * kApThreads + tid;
    if (v >= nv) continue;
    const uint32_t a[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
    uint32_t o[2] = {0, 0};
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      const float f = __uint_as_float((t & 1) ? a[t >> 1] & 0xffff0000u : a[t >> 1] << 16);
      const float u = fminf(fmaxf(pow2 ? f * inv : f / scale, -most), most);
      o[t >> 2] |= quant_byte(u, FMT) << (8 * (t & 3));
    }
    reinterpret_cast<uint2*>(codes + static_cast<int64_t>(lo) * D)[v] = make_uint2(o[0], o[1]);
  }
  if (tid == 0) p.scale[kv][tile] = scale;
}

template <int FMT, int D>
void launch_append(const AppendParams& p, dim3 grid, cudaStream_t s) {
  k_kv8_append<FMT, D><<<grid, kApThreads, 0, s>>>(p);
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
  p.src[0] = static_cast<const __nv_bfloat16*>(k), p.src[1] = static_cast<const __nv_bfloat16*>(v);
  p.stride[0] = k_stride, p.stride[1] = v_stride;
  p.dst[0] = static_cast<uint8_t*>(cache->k), p.dst[1] = static_cast<uint8_t*>(cache->v);
  p.scale[0] = cache->k_scale, p.scale[1] = cache->v_scale;
  p.seqs = {seqs->cu_q, seqs->kv_lens, seqs->block_table, seqs->T, seqs->B, seqs->max_q, seqs->max_blocks};
  p.num_blocks = cache->num_blocks, p.block = cache->block, p.heads = cache->kv_heads;
  p.status = static_cast<int32_t*>(status);
  // n new tokens touch at most (n - 1) / block + 2 blocks, and never more than
  // n; so the batch at most the sum of either over its sequences
  long long most = seqs->T / cache->block + 2ll * seqs->B;
  if (most > seqs->T) most = seqs->T;
  if (most > 0x7fffffffll) return FL_ERR_UNSUPPORTED;
  const dim3 grid(static_cast<unsigned>(most), cache->kv_heads, 2);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (cache->format == FL_KV8_E4M3)
    cache->head_dim == 64 ? launch_append<FL_KV8_E4M3, 64>(p, grid, s) : launch_append<FL_KV8_E4M3, 128>(p, grid, s);
  else
    cache->head_dim == 64 ? launch_append<FL_KV8_INT8, 64>(p, grid, s) : launch_append<FL_KV8_INT8, 128>(p, grid, s);
  return cudaGetLastError() == cudaSuccess ? FL_OK : FL_ERR_CUDA;
}

extern "C" int fl_kv8_test_pages(const fl_kv8_seqs* seqs, int num_blocks, int block, int window, int b, long long* out) {
  if (!seqs || !out || !seqs->kv_lens || !seqs->block_table || num_blocks < 1 || block < 1 || window < 0 || b < 0 ||
      b >= seqs->B || seqs->T > (1 << 29) || seqs->max_blocks > (1 << 30) / block)
    return FL_ERR_ARG;
  if (window >= seqs->max_blocks * block) window = 0;
  const Seqs s = {seqs->cu_q, seqs->kv_lens, seqs->block_table, seqs->T, seqs->B, seqs->max_q, seqs->max_blocks};
  const SeqInfo q = seq_info(s, b, block);
  const PageRun runs[2] = {written_pages(q, block), read_pages(q, block, window)};
  out[0] = q.start, out[1] = q.n, out[2] = q.kv;
  for (int i = 0; i < 2; ++i) {
    out[3 + 3 * i] = runs[i].first, out[4 + 3 * i] = runs[i].n, out[5 + 3 * i] = 0;
    for (int pg = 0; pg < runs[i].n; ++pg) out[5 + 3 * i] += page_block(s, b, runs[i].first + pg, num_blocks) < 0;
  }
  return FL_OK;
}
