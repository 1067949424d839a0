// The split of a prompt's attention into units, and the launch of its kernel.
#pragma once

#include <cuda.h>

#include "fl_kv8.cuh"

namespace flkv {

constexpr int kPromptRows = 256;   // rows of an item: two row tiles of 128
constexpr int kPromptTile = 128;   // tokens of a unit

// sum over i < n of floor((a i + b) / m), for n >= 0, m >= 1, a, b >= 0 and
// sums, on the way too, within 32 bits
__host__ __device__ __forceinline__ unsigned floor_sum(unsigned n, unsigned m, unsigned a, unsigned b) {
  unsigned sum = 0;
  while (n > 0) {
    const unsigned qa = a / m, qb = b / m;
    sum += n * (n - 1) / 2 * qa + n * qb;
    a -= qa * m;
    b -= qb * m;
    const unsigned y = a * n + b;
    if (y < m) break;
    n = y / m;
    b = y - n * m;
    const unsigned t = m;
    m = a;
    a = t;
  }
  return sum;
}

// The units of one sequence: items (kv head, 256 rows) of `tiles(i)` units
// each, a unit one tile of 128 tokens.  Rows are token-major (token, query
// head of the group).  A causal sequence's item i ends with the tile of its
// last row's own position, so that its tiles are those that some row sees:
//   tiles(i) = floor((past g + 256 (i + 1) - 1) / (128 g)) + 1,
// summed in closed form (the division by 128 g is one by 128, then one by g).
// With a window, with rows before the first token, or with sums past 32 bits,
// every item gets the same number of units, some of them without work.
struct PromptWork {
  SeqInfo q;
  int rows, items, g, past, window, nc;   // nc: units of each item, 0 for the causal form
  long long per_head;

  __host__ __device__ long long before(int i) const {   // units of a head's items before item i
    if (nc) return static_cast<long long>(i) * nc;
    const int k = min(i, items - 1);
    const unsigned b = static_cast<unsigned>((static_cast<long long>(past) * g + 255) >> 7);
    const long long n = k + static_cast<long long>(floor_sum(k, g, 2, b));
    return i < items ? n : n + (q.kv + kPromptTile - 1) / kPromptTile;
  }
  __host__ __device__ int tiles(int i) const { return static_cast<int>(before(i + 1) - before(i)); }
  __host__ __device__ int item_of(long long u) const {   // the item that unit u of a head lies in
    int lo = 0, hi = items - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (before(mid) <= u)
        lo = mid;
      else
        hi = mid - 1;
    }
    return lo;
  }
  // Tokens [low, lim) that some row of [r0, r0 + n) sees (lim <= low: none).
  __host__ __device__ int lim(int r0, int n) const { return past + min(r0 + n - 1, rows - 1) / g + 1; }
  __host__ __device__ int low(int r0) const { return window ? max(0, past + r0 / g + 1 - window) : 0; }
  __host__ __device__ int first_tile(int i) const { return low(i * kPromptRows) / kPromptTile; }
};

__host__ __device__ __forceinline__ PromptWork prompt_work(const SeqInfo& q, int group, int heads, int window, int rows_lo,
                                                           int rows_hi) {
  PromptWork w;
  w.q = q;
  w.g = group;
  w.rows = q.n * group;
  w.items = w.rows > rows_lo && w.rows <= rows_hi ? (w.rows + kPromptRows - 1) / kPromptRows : 0;
  w.past = q.kv - q.n;
  w.window = window < q.kv ? window : 0;
  w.nc = 0;
  // The sums of the causal form have to fit 32 bits: items^2 is below 2^30,
  // items times a quotient of at most kv / 128 + 3 too, 2 items + b below 2^31.
  const bool fits = w.items < 32768 && static_cast<long long>(w.items) * (q.kv / kPromptTile + 3) < (1ll << 30) &&
                    static_cast<long long>(q.kv) * group < (1ll << 36);
  if (w.past < 0 || w.window || !fits) {
    const int all = max(1, (q.kv + kPromptTile - 1) / kPromptTile);
    // a window's first tile starts up to 127 tokens early, and an item's rows
    // span up to 256 / g + 1 tokens
    const int win = w.window ? (w.window + kPromptRows / group + 1) / kPromptTile + 2 : all;
    w.nc = min(all, win);
  }
  w.per_head = w.items ? w.before(w.items) : 0;
  return w;
}

int launch_prompt(const CUtensorMap& km, const CUtensorMap& vm, const AttnParams& p, int format, int head_dim, cudaStream_t s);
size_t prompt_scratch(int head_dim);   // bytes of partials

}  // namespace flkv
