// Book-keeping of the 8-bit cache's pages on the device: giving pages back,
// sharing them, finding free ones, moving the ones in use together, and the
// copies that follow.
//
// free and fork take a CTA a sequence; counts of holders are integer atomics,
// whose order does not matter.  alloc and compact decide in list order, so one
// CTA scans the list and the pool with prefix sums: with 1024 threads 4096
// counts a step, and no more of the pool than the pages that are wanted.  They are
// bound by latency: a dozen dependent loads and barriers.  The copy moves 16-byte
// vectors, eight in flight a thread, over a grid that fills the GPU; it is bound by
// HBM: every byte of a page once in and once out.  Compacting a pool of 9001 pages
// of 256 KB, 2160 of which move, takes 196 us, 186 of them the copy (6.1 TB/s).
#include <limits>

#include "fl_common.cuh"

using namespace fl;

namespace {

constexpr int kScanThreads = 1024;
constexpr int kListThreads = 128;

struct Pool {
  int32_t* refs;
  int32_t* table;
  int32_t* lens;
  int blocks, slots, most, block;
  __device__ __forceinline__ int32_t* row(int s) const { return table + static_cast<int64_t>(s) * most; }
  __device__ __forceinline__ int pages(int tokens) const { return static_cast<int>((tokens + block - 1ll) / block); }
  __device__ __forceinline__ bool page(int id) const { return id >= 0 && id < blocks; }
};

__device__ void missing(int32_t* status, int detail) { set_status(status, FL_ERR_DEVICE_CHECK, detail); }

// Sum over the block (all threads call it), and this thread's sum of those before it.
__device__ __forceinline__ long long scan_block(long long v, long long* all) {
  __shared__ long long sums[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long inc = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, inc, d);
    if (lane >= d) inc += u;
  }
  __syncthreads();   // (the sums of the scan before have been read)
  if (lane == 31) sums[warp] = inc;
  __syncthreads();
  long long w = lane < blockDim.x / 32 ? sums[lane] : 0;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, w, d);
    if (lane >= d) w += u;
  }
  *all = __shfl_sync(0xffffffffu, w, 31);
  const long long before = __shfl_sync(0xffffffffu, w, warp ? warp - 1 : 0);
  return (warp ? before : 0) + inc - v;
}

// ------------------------------------------------------------------- free
__global__ void __launch_bounds__(kListThreads) k_pages_free(const Pool p, const int32_t* seqs, const int32_t* keep, int32_t* status) {
  __shared__ int was;
  pdl_wait();
  pdl_launch_dependents();
  const int s = seqs[blockIdx.x];
  if (s < 0 || s >= p.slots) {
    if (threadIdx.x == 0) missing(status, 70);
    return;
  }
  const int left = keep ? max(keep[blockIdx.x], 0) : 0;
  // the slot may be in the list again: the length only falls, and an entry is
  // taken out of the table once, whoever comes first
  if (threadIdx.x == 0) was = atomicMin(p.lens + s, left);
  __syncthreads();
  const int end = min(p.pages(max(was, 0)), p.most);
  for (int j = p.pages(left) + threadIdx.x; j < end; j += kListThreads) {
    const int id = atomicExch(p.row(s) + j, -1);
    if (id == -1) continue;
    if (!p.page(id)) {
      missing(status, 71);
    } else if (atomicAdd(p.refs + id, -1) <= 0) {
      atomicAdd(p.refs + id, 1);
      missing(status, 72);
    }
  }
}

// ------------------------------------------------------------------- fork
__global__ void __launch_bounds__(kListThreads) k_pages_fork(const Pool p, const int32_t* parents, const int32_t* children, int n,
                                                             int32_t* status) {
  pdl_wait();
  pdl_launch_dependents();
  const int i = blockIdx.x, from = parents[i], to = children[i];
  bool bad = from < 0 || from >= p.slots || to < 0 || to >= p.slots;
  for (int j = threadIdx.x; j < n; j += kListThreads) bad |= parents[j] == to || (j < i && children[j] == to);
  if (!bad && threadIdx.x == 0) bad = p.lens[to] != 0 || p.lens[from] < 0 || p.lens[from] > static_cast<long long>(p.most) * p.block;
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0) missing(status, 73);
    return;
  }
  // (a parent is no child of the list: its length and pages stand still)
  const int len = p.lens[from], pages = p.pages(len);
  for (int j = threadIdx.x; j < pages; j += kListThreads) {
    const int id = p.row(from)[j];
    p.row(to)[j] = id;
    if (p.page(id))
      atomicAdd(p.refs + id, 1);
    else
      missing(status, 74);
  }
  if (threadIdx.x == 0) p.lens[to] = len;
}

// ------------------------------------------------------------------ alloc
struct AllocParams {
  Pool p;
  const int32_t* seqs;
  const int32_t* wanted;
  int n;
  int32_t* granted;
  int32_t* pairs;
  int32_t* count;
  int32_t* first;     // [slots] the list entry that names the slot first
  int32_t* sharers;   // [blocks] entries that would write into the page
  int32_t* last;      // [blocks] the last of them
  int32_t* free;      // [blocks] free pages, ascending
  int32_t* status;
};

// What entry i of the list asks for; page -1: no page that it may share.
struct Ask {
  int slot, old, end, page;
  bool ok;
};
__device__ __forceinline__ Ask ask(const AllocParams& a, int i) {
  const Pool& p = a.p;
  Ask r = {a.seqs[i], 0, 0, -1, false};
  if (r.slot < 0 || r.slot >= p.slots) {
    r.slot = -1;
    return r;
  }
  const int add = a.wanted[i];
  r.old = p.lens[r.slot];
  const long long end = static_cast<long long>(r.old) + add;
  if (add < 0 || r.old < 0 || end > static_cast<long long>(p.most) * p.block || end > 0x7fffffffll - p.block) return r;
  r.end = static_cast<int>(end);
  if (r.old % p.block && add) {
    r.page = p.row(r.slot)[r.old / p.block];
    if (!p.page(r.page)) {
      r.page = -1;
      return r;
    }
  }
  r.ok = true;
  return r;
}

__global__ void __launch_bounds__(kScanThreads) k_pages_alloc(const AllocParams a) {
  const Pool& p = a.p;
  const int tid = threadIdx.x, lane = tid & 31;
  pdl_wait();
  pdl_launch_dependents();
  for (int i = tid; i < a.n; i += kScanThreads) {
    const Ask q = ask(a, i);
    if (q.slot >= 0) a.first[q.slot] = std::numeric_limits<int>::max();
    if (q.page >= 0) a.sharers[q.page] = 0, a.last[q.page] = -1;
  }
  __syncthreads();
  for (int i = tid; i < a.n; i += kScanThreads) {
    const int s = a.seqs[i];
    if (s >= 0 && s < p.slots) atomicMin(a.first + s, i);
  }
  __syncthreads();
  for (int i = tid; i < a.n; i += kScanThreads) {
    const Ask q = ask(a, i);
    if (q.ok && q.page >= 0 && __ldcg(a.first + q.slot) == i) {
      atomicAdd(a.sharers + q.page, 1);
      atomicMax(a.last + q.page, i);
    }
  }
  __syncthreads();
  // granted[i] holds the entry's new pages and whether one is a copy, until all are known
  long long total = 0;
  for (int i = tid; i < a.n; i += kScanThreads) {
    const Ask q = ask(a, i);
    int got = -1;
    if (q.ok && __ldcg(a.first + q.slot) == i) {
      const int refs = q.page >= 0 ? p.refs[q.page] : 0;
      const bool copy = refs > 1 && !(__ldcg(a.sharers + q.page) == refs && __ldcg(a.last + q.page) == i);
      const int need = p.pages(q.end) - p.pages(q.old) + copy;
      got = 2 * need + copy;
      total += need;
    } else {
      missing(a.status, 75);
    }
    a.granted[i] = got;
  }
  long long all;
  scan_block(total, &all);
  total = all;
  // the first free pages, as many as are wanted
  long long found = 0;
  for (int at = 0; at < p.blocks && found < total; at += 4 * kScanThreads) {
    int r[4], n = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int id = at + 4 * tid + e;
      r[e] = id < p.blocks && p.refs[id] <= 0;
      n += r[e];
    }
    long long k = found + scan_block(n, &all);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (r[e]) a.free[k++] = at + 4 * tid + e;
    found += all;
  }
  __syncthreads();
  // grants, in list order
  long long taken = 0, copies = 0;
  for (int i0 = 0; i0 < a.n; i0 += kScanThreads) {
    const int i = i0 + tid, got = i < a.n ? a.granted[i] : -1;
    const int need = got >= 0 ? got >> 1 : 0;
    int copy = got >= 0 ? got & 1 : 0;
    const long long before = taken + scan_block(need, &all);
    taken += all;
    const bool ok = got >= 0 && before + need <= found;
    copy = ok ? copy : 0;
    const long long rank = copies + scan_block(copy, &all);
    copies += all;
    Ask q = {0, 0, 0, -1, false};
    if (ok) q = ask(a, i);
    const int start = ok ? (copy ? q.old / p.block : p.pages(q.old)) : 0;
    __syncwarp();
    if (i < a.n) a.granted[i] = ok;
    if (copy) {
      a.pairs[2 * rank] = q.page, a.pairs[2 * rank + 1] = a.free[before];
      atomicAdd(p.refs + q.page, -1);
    }
    // few pages by the entry's thread, many by its warp
    const bool many = ok && need > 4;
    if (ok && !many)
      for (int j = 0; j < need; ++j) {
        const int id = a.free[before + j];
        p.row(q.slot)[start + j] = id;
        p.refs[id] = 1;
      }
    for (uint32_t left = __ballot_sync(0xffffffffu, many); left; left &= left - 1) {
      const int src = __ffs(left) - 1;
      const int n = __shfl_sync(0xffffffffu, need, src), slot = __shfl_sync(0xffffffffu, q.slot, src);
      const int s = __shfl_sync(0xffffffffu, start, src);
      const long long b = __shfl_sync(0xffffffffu, before, src);
      for (int j = lane; j < n; j += 32) {
        const int id = a.free[b + j];
        p.row(slot)[s + j] = id;
        p.refs[id] = 1;
      }
    }
    if (ok) p.lens[q.slot] = q.end;
  }
  if (tid == 0) *a.count = static_cast<int>(copies);
  for (long long i = copies + tid; i < a.n; i += kScanThreads) a.pairs[2 * i] = a.pairs[2 * i + 1] = -1;
}

// ---------------------------------------------------------------- compact
struct CompactParams {
  Pool p;
  int32_t* table;
  int32_t* refs;
  int32_t* moved;
  int32_t* pairs;
  int32_t* count;
  int32_t* status;
};

__global__ void __launch_bounds__(kScanThreads) k_pages_compact(const CompactParams c) {
  const Pool& p = c.p;
  const int tid = threadIdx.x;
  pdl_wait();
  pdl_launch_dependents();
  long long live = 0, all;
  for (int i = tid; i < p.blocks; i += kScanThreads) live += p.refs[i] > 0;
  scan_block(live, &all);
  const int n = static_cast<int>(all);
  // the k-th page in use from n on and the k-th free one before n make pair k:
  // there are as many of the one as of the other
  long long highs = 0, holes = 0;
  for (int at = 0; at < p.blocks; at += 4 * kScanThreads) {
    int r[4];
    long long v = 0;   // highs above, holes below
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int id = at + 4 * tid + e;
      r[e] = id < p.blocks ? p.refs[id] : 0;
      if (id < p.blocks) v += r[e] > 0 ? (id >= n ? 1ll << 32 : 0) : (id < n ? 1 : 0);
    }
    const long long before = scan_block(v, &all);
    long long high = highs + (before >> 32), hole = holes + (before & 0xffffffffll);
    highs += all >> 32, holes += all & 0xffffffffll;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int id = at + 4 * tid + e;
      if (id >= p.blocks) continue;
      if (r[e] > 0) {
        if (id >= n) c.pairs[2 * high++] = id;
        c.moved[id] = id;
      } else {
        if (id < n) c.pairs[2 * hole++ + 1] = id;
        c.moved[id] = -1;
      }
      if (c.refs != p.refs) c.refs[id] = r[e];
    }
  }
  __syncthreads();
  for (int k = tid; k < highs; k += kScanThreads) {
    const int from = c.pairs[2 * k], to = c.pairs[2 * k + 1];
    c.moved[from] = to;
    c.refs[to] = c.refs[from];
    c.refs[from] = 0;
  }
  for (int k = static_cast<int>(highs) + tid; k < p.blocks / 2; k += kScanThreads) c.pairs[2 * k] = c.pairs[2 * k + 1] = -1;
  if (tid == 0) *c.count = static_cast<int>(highs);
}

// The table's entries after the moves.
__global__ void __launch_bounds__(256) k_pages_table(const CompactParams c) {
  const Pool& p = c.p;
  pdl_wait();
  pdl_launch_dependents();
  const long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= static_cast<long long>(p.slots) * p.most) return;
  const int s = static_cast<int>(i / p.most), j = static_cast<int>(i - static_cast<long long>(s) * p.most);
  int id = p.table[i];
  if (j < p.pages(max(p.lens[s], 0))) {
    const int to = p.page(id) ? c.moved[id] : -1;
    if (to < 0) missing(c.status, 76);
    id = to;
  }
  c.table[i] = id;
}

// ------------------------------------------------------------------- copy
constexpr int kLayers = 64;           // caches of one launch
constexpr int kCopyThreads = 256;
constexpr int kCopyVecs = 8;          // 16-byte vectors of a thread and step

struct CopyParams {
  uint8_t* codes[kLayers][2];
  float* scales[kLayers][2];
  const int32_t* pairs;
  const int32_t* count;
  int32_t* status;
  int layers, max_pairs, blocks, heads;
  int page_vecs;   // 16-byte vectors of a page's keys
};

__global__ void __launch_bounds__(kCopyThreads) k_pages_copy(const __grid_constant__ CopyParams p) {
  pdl_wait();
  pdl_launch_dependents();
  const int n = min(max(*p.count, 0), p.max_pairs);
  constexpr int kStep = kCopyThreads * kCopyVecs;
  const int steps = (p.page_vecs + kStep - 1) / kStep, halves = 2 * p.layers;
  const long long items = static_cast<long long>(n) * halves * steps;
  for (long long it = blockIdx.x; it < items; it += gridDim.x) {
    const int step = static_cast<int>(it % steps);
    const long long h = it / steps;
    const int half = static_cast<int>(h % halves), pair = static_cast<int>(h / halves);
    const int from = p.pairs[2 * pair], to = p.pairs[2 * pair + 1];
    if (from < 0 || from >= p.blocks || to < 0 || to >= p.blocks) {
      if (threadIdx.x == 0) missing(p.status, 77);
      continue;
    }
    const uint4* src = reinterpret_cast<const uint4*>(p.codes[half >> 1][half & 1]) + static_cast<int64_t>(from) * p.page_vecs;
    uint4* dst = reinterpret_cast<uint4*>(p.codes[half >> 1][half & 1]) + static_cast<int64_t>(to) * p.page_vecs;
    const int at = step * kStep + threadIdx.x;
    uint4 v[kCopyVecs];
#pragma unroll
    for (int i = 0; i < kCopyVecs; ++i)
      if (at + i * kCopyThreads < p.page_vecs) v[i] = __ldcs(src + at + i * kCopyThreads);
#pragma unroll
    for (int i = 0; i < kCopyVecs; ++i)
      if (at + i * kCopyThreads < p.page_vecs) __stcs(dst + at + i * kCopyThreads, v[i]);
    if (step == 0) {
      float* sc = p.scales[half >> 1][half & 1];
      for (int i = threadIdx.x; i < p.heads; i += kCopyThreads)
        sc[static_cast<int64_t>(to) * p.heads + i] = sc[static_cast<int64_t>(from) * p.heads + i];
    }
  }
}

// ------------------------------------------------------------------- host
bool word(const void* p) { return p && reinterpret_cast<uintptr_t>(p) % 4 == 0; }

int check_pool(const fl_kv8_pool* p) {
  if (!p || !word(p->refs) || !word(p->table) || !word(p->kv_lens) || p->num_blocks < 1 || p->slots < 1 || p->max_blocks < 1)
    return FL_ERR_ARG;
  if (p->block != 16 && p->block != 32 && p->block != 64 && p->block != 128) return FL_ERR_UNSUPPORTED;
  if (static_cast<long long>(p->slots) * p->max_blocks > 0x7fffffffll || p->num_blocks > (1 << 30)) return FL_ERR_UNSUPPORTED;
  return FL_OK;
}
Pool view(const fl_kv8_pool& p) { return {p.refs, p.table, p.kv_lens, p.num_blocks, p.slots, p.max_blocks, p.block}; }
cudaStream_t stream_of(fl_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

struct AllocLayout {
  size_t first, sharers, last, free, bytes;
};
AllocLayout alloc_layout(const fl_kv8_pool& p) {
  AllocLayout l;
  auto up = [](size_t v) { return (v + 255) / 256 * 256; };
  const size_t blocks = up(static_cast<size_t>(p.num_blocks) * 4);
  l.first = kScratchOff;
  l.sharers = l.first + up(static_cast<size_t>(p.slots) * 4);
  l.last = l.sharers + blocks;
  l.free = l.last + blocks;
  l.bytes = l.free + blocks;
  return l;
}

}  // namespace

extern "C" int fl_kv8_pages_free(const fl_kv8_pool* pool, const int32_t* seqs, const int32_t* keep, int n, void* status,
                                 fl_stream_t stream) {
  const int rc = check_pool(pool);
  if (rc != FL_OK) return rc;
  if (n < 0 || (n && !word(seqs)) || (keep && !word(keep)) || !status || !flh::aligned16(status)) return FL_ERR_ARG;
  if (n == 0) return FL_OK;
  return flh::launch_early(k_pages_free, dim3(n), dim3(kListThreads), 0, stream_of(stream), view(*pool), seqs, keep,
                           static_cast<int32_t*>(status));
}

extern "C" int fl_kv8_pages_fork(const fl_kv8_pool* pool, const int32_t* parents, const int32_t* children, int n, void* status,
                                 fl_stream_t stream) {
  const int rc = check_pool(pool);
  if (rc != FL_OK) return rc;
  if (n < 0 || (n && (!word(parents) || !word(children))) || !status || !flh::aligned16(status)) return FL_ERR_ARG;
  if (n == 0) return FL_OK;
  return flh::launch_early(k_pages_fork, dim3(n), dim3(kListThreads), 0, stream_of(stream), view(*pool), parents, children, n,
                           static_cast<int32_t*>(status));
}

extern "C" int fl_kv8_pages_workspace(const fl_kv8_pool* pool, size_t* out) {
  const int rc = check_pool(pool);
  if (rc != FL_OK) return rc;
  if (!out) return FL_ERR_ARG;
  *out = alloc_layout(*pool).bytes;
  return FL_OK;
}

extern "C" int fl_kv8_pages_alloc(const fl_kv8_pool* pool, const int32_t* seqs, const int32_t* new_tokens, int n, int32_t* granted,
                                  int32_t* pairs, int32_t* count, void* ws, size_t ws_bytes, fl_stream_t stream) {
  const int rc = check_pool(pool);
  if (rc != FL_OK) return rc;
  if (n < 0 || n > (1 << 30) || !word(count) || !ws || !flh::aligned16(ws)) return FL_ERR_ARG;
  if (n && (!word(seqs) || !word(new_tokens) || !word(granted) || !word(pairs))) return FL_ERR_ARG;
  const AllocLayout l = alloc_layout(*pool);
  if (ws_bytes < l.bytes) return FL_ERR_WORKSPACE;
  uint8_t* base = static_cast<uint8_t*>(ws);
  auto ints = [&](size_t at) { return reinterpret_cast<int32_t*>(base + at); };
  const AllocParams a = {view(*pool), seqs, new_tokens, n, granted, pairs, count, ints(l.first), ints(l.sharers), ints(l.last),
                         ints(l.free), ints(0)};
  return flh::launch_early(k_pages_alloc, dim3(1), dim3(kScanThreads), 0, stream_of(stream), a);
}

extern "C" int fl_kv8_pages_compact(const fl_kv8_pool* pool, int32_t* table_out, int32_t* refs_out, int32_t* moved, int32_t* pairs,
                                    int32_t* count, void* status, fl_stream_t stream) {
  const int rc = check_pool(pool);
  if (rc != FL_OK) return rc;
  if (!word(table_out) || !word(refs_out) || !word(moved) || (!word(pairs) && pool->num_blocks > 1) || !word(count) || !status ||
      !flh::aligned16(status))
    return FL_ERR_ARG;
  const CompactParams c = {view(*pool), table_out, refs_out, moved, pairs, count, static_cast<int32_t*>(status)};
  const int r = flh::launch_early(k_pages_compact, dim3(1), dim3(kScanThreads), 0, stream_of(stream), c);
  if (r != FL_OK) return r;
  const long long entries = static_cast<long long>(pool->slots) * pool->max_blocks;
  return flh::launch_early(k_pages_table, dim3(static_cast<unsigned>((entries + 255) / 256)), dim3(256), 0, stream_of(stream), c);
}

extern "C" int fl_kv8_pages_copy(const fl_kv8_cache* caches, int layers, const int32_t* pairs, const int32_t* count, int max_pairs,
                                 void* status, fl_stream_t stream) {
  if (!caches || layers < 1 || max_pairs < 0 || (max_pairs && !word(pairs)) || !word(count) || !status || !flh::aligned16(status))
    return FL_ERR_ARG;
  const fl_kv8_cache& c = caches[0];
  if (c.num_blocks < 1 || c.kv_heads < 1) return FL_ERR_ARG;
  if ((c.block != 16 && c.block != 32 && c.block != 64 && c.block != 128) || (c.head_dim != 64 && c.head_dim != 128)) return FL_ERR_UNSUPPORTED;
  const long long tokens = static_cast<long long>(c.kv_heads) * c.block;
  if (tokens * c.num_blocks > 0x7fffffffll || tokens * c.head_dim > 0x7fffffffll) return FL_ERR_UNSUPPORTED;
  for (int i = 0; i < layers; ++i) {
    const fl_kv8_cache& d = caches[i];
    if (!d.k || !d.v || !flh::aligned16(d.k) || !flh::aligned16(d.v) || !word(d.k_scale) || !word(d.v_scale)) return FL_ERR_ARG;
    if (d.num_blocks != c.num_blocks || d.block != c.block || d.kv_heads != c.kv_heads || d.head_dim != c.head_dim) return FL_ERR_ARG;
  }
  if (max_pairs == 0) return FL_OK;
  CopyParams p;
  p.pairs = pairs, p.count = count, p.status = static_cast<int32_t*>(status);
  p.max_pairs = max_pairs, p.blocks = c.num_blocks, p.heads = c.kv_heads;
  p.page_vecs = static_cast<int>(tokens * c.head_dim / 16);
  constexpr int kStep = kCopyThreads * kCopyVecs;
  for (int i = 0; i < layers; i += kLayers) {
    p.layers = layers - i < kLayers ? layers - i : kLayers;
    for (int j = 0; j < p.layers; ++j) {
      const fl_kv8_cache& d = caches[i + j];
      p.codes[j][0] = static_cast<uint8_t*>(d.k), p.codes[j][1] = static_cast<uint8_t*>(d.v);
      p.scales[j][0] = d.k_scale, p.scales[j][1] = d.v_scale;
    }
    const long long items = static_cast<long long>(max_pairs) * 2 * p.layers * ((p.page_vecs + kStep - 1) / kStep);
    const long long grid = items < 8ll * flh::sm_count() ? items : 8ll * flh::sm_count();
    const int rc = flh::launch_early(k_pages_copy, dim3(static_cast<unsigned>(grid)), dim3(kCopyThreads), 0, stream_of(stream), p);
    if (rc != FL_OK) return rc;
  }
  return FL_OK;
}
