// What the kernels of medusa_linear_w4 share.
#pragma once

#include "common.cuh"

namespace medusa {
namespace w4 {

struct Args {
  const uint16_t* x;
  long long ldx;
  const uint32_t* q;
  const uint16_t* scales;
  const uint8_t* zeros;
  int T, K, Nout, glog;  // glog: log2 of the group
  void* y;
  int y32;
  int32_t* d_status;
};

__device__ __forceinline__ uint32_t sub2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// What a group's weights are made of: 128 + zero and the scale, twice each.
struct Group {
  uint32_t base, scale;
};
__device__ __forceinline__ Group group_of(uint32_t scale, uint32_t zero) {
  const uint32_t b = 0x4300u | (zero & 127u);
  return {b | b << 16, scale | scale << 16};
}
__device__ __forceinline__ Group group_at(const Args& a, int g, int n) {
  const size_t i = (size_t)g * a.Nout + n;
  return group_of(a.scales[i], a.zeros ? a.zeros[i] : 8);
}
// The four pairs of a word.  The three-operand logic operation takes one immediate: with both constants written
// out it became two operations, a fifth of all.
__device__ __forceinline__ uint32_t nibbles(uint32_t w, uint32_t magic) {
  uint32_t r;
  asm("lop3.b32 %0, %1, 0x000f000f, %2, 0xea;" : "=r"(r) : "r"(w), "r"(magic));
  return r;
}
__device__ __forceinline__ void unpack(uint32_t w, const Group& g, uint32_t* p) {
  uint32_t magic;
  asm("mov.b32 %0, 0x43004300;" : "=r"(magic));
#pragma unroll
  for (int i = 0; i < 4; ++i) p[i] = mul2(sub2(nibbles(w >> (4 * i), magic), g.base), g.scale);
}

// To bf16, to nearest even, by the hardware's conversion.
__device__ __forceinline__ uint16_t bf16_rn(float v) {
  uint16_t r;
  asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ void store_y(const Args& a, int t, int n, float v) {
  const size_t i = (size_t)t * a.Nout + n;
  if (a.y32) static_cast<float*>(a.y)[i] = v;
  else static_cast<uint16_t*>(a.y)[i] = bf16_rn(v);
}

// Clusters of `share` CTAs of a tensor-memory kernel, one CTA an SM, that the current device holds at once.
int clusters_at_once(int share);
// Tensor-memory kernels: few tokens or a small layer (linear_w4_stream.cu), any number (linear_w4_tc.cu).
medusa_status stream_launch(const Args& a, int withhold, cudaStream_t s);
// Blocks of 128 features, 64 tokens and 128 columns that a CTA of the first one has at most.
int stream_blocks(int T, int K, int Nout);
medusa_status tc_launch(const Args& a, int withhold, cudaStream_t s);
// How a kernel divides a layer, for tests.
struct Division {
  int share, tokens, features, tiles, ctas;  // CTAs that share a tile; of a tile; all of them
};
Division stream_division(int T, int K, int Nout);
Division tc_division(int T, int K, int Nout);

}  // namespace w4
}  // namespace medusa
