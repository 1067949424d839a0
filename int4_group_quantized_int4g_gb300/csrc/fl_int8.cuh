// Shared pieces of the linear layer in 8-bit integers.
#pragma once

#include "fl_tc.cuh"

namespace fl8 {

using namespace fl;

constexpr int kBlockK = 128;      // columns of a work unit
constexpr int kRowsMax = 16;      // tokens of the streaming kernel: with 24 the head of 128003 takes 102 us there, 90 on tcgen05
constexpr size_t kScratch = kScratchOff;   // status and counters before it, as in every workspace

// Four codes of a word as two f16 pairs, exactly: f16 1024 + u holds the byte u
// in its last bits, and u = code + 128.
__device__ __forceinline__ void codes_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  const uint32_t u = w ^ 0x80808080u;
  const __half2 bias = __half2half2(__ushort_as_half(0x6480));   // 1152
  const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140u), b = __byte_perm(u, 0x64646464u, 0x4342u);
  const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&a), bias);
  const __half2 y = __hsub2(*reinterpret_cast<const __half2*>(&b), bias);
  lo = *reinterpret_cast<const uint32_t*>(&x);
  hi = *reinterpret_cast<const uint32_t*>(&y);
}

// Where each part of a call's scratch begins.
struct Layout {
  size_t scale, x, part, bytes;
};

// One linear call, after x has become f16 codes in the workspace.
struct Call {
  const void* xh;          // f16 codes: rows of K, or fragments (M <= kRowsMax)
  const float* x_scale;
  const int8_t* w;
  const float* w_scale;
  void* y;
  int64_t y_stride;
  float* part;
  int32_t* cnt;
  int32_t* status;
  int M, K, N, fp32;
};

int rows_launch(const Call& c, cudaStream_t s);
size_t rows_part_bytes(int M);
int gemm_launch(const Call& c, cudaStream_t s);
// How the tiles of 256 weight rows x BN tokens (G units of 128 columns each) go to P
// pairs of SMs: `waves` whole ones each, and `units` of the rest, first, in equal runs
// or (whole) a tile for each of the first pairs.
struct Plan {
  int BN, G;
  long long mtiles, ntiles;
  int P, waves;
  long long units;
  int whole;
};
Plan gemm_plan(int M, int N, int K, int pairs);
size_t gemm_part_bytes(int M, int N, int K);

}  // namespace fl8
