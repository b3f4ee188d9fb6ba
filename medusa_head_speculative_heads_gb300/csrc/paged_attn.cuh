// What the two paged-attention kernels (CUDA cores and tensor cores) and the
// merge of their partial results share.
#pragma once

#include <cuda_runtime.h>

#include "medusa.h"
#include "paged.cuh"

namespace medusa {
namespace paged {

// What the merge of a CTA boundary needs: the item the boundary falls inside,
// and the CTAs that have its parts.  first < 0: nothing, or an earlier
// boundary's.
struct __align__(16) Shared {
  Item it;
  int first, last;
};

// Two fp32 operations at once.
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

struct AttnArgs {
  Work w;
  Cache cache;
  const void *q, *k_pages, *v_pages, *kt, *vt;
  const uint32_t* mask;  // [N][W]
  void* out;
  float* lse;
  float* part_o;    // [slot][R / rows of a group][d / 4][row][4]: unnormalised sums of shared items
  float2* part_ml;  // [slot][R] their row maxima (log2 domain) and row sums
  Shared* shared;   // [CTA] the boundary its range starts at
  int32_t* d_status;
  long long ldq;
  int Hq, Hkv, d, G;
  int sub, nsub;  // q heads per head group, groups per kv head
  int R;          // rows of a partial slot
  int tile_rows, tile_tok;  // a block is tiles of tile_rows rows: tile_tok tokens x sub heads each
  int W;
  int withhold;  // failure test: the tensor-core kernel brings no V
  int out32;  // rows of out start on 32 bytes
  float scale_log2;
};

// Row r of item it's block: its token within the sequence and its q head.
struct Row {
  int tok, h;
  bool ok;
};
__device__ __forceinline__ Row row_of(const AttnArgs& a, const Item& it, int r) {
  Row x;
  const int tile = r / a.tile_rows, m = r - tile * a.tile_rows;
  const int t = m / a.sub, g = m - t * a.sub;
  const int hg = it.lg % a.w.nh, part = hg % a.nsub;
  x.tok = it.i * a.w.ctok + tile * a.tile_tok + t;
  x.h = hg / a.nsub * a.G + part * a.sub + g;
  x.ok = t < a.tile_tok && x.tok < it.s.len && part * a.sub + g < a.G;
  return x;
}
// Index of the row in q, out ([nl * T] tokens, Hq heads) and lse.
__device__ __forceinline__ size_t out_row(const AttnArgs& a, const Item& it, const Row& x) {
  return ((size_t)(it.lg / a.w.nh) * a.w.T + it.s.q0 + x.tok) * a.Hq + x.h;
}

// Rows whose fours of columns take turns in a partial slot.  Of a big slot a warp's
// worth: lanes that hold a row each then write and read neighbouring words (a
// store of 32 separate lines takes 32 clocks).  Of a small one, in which few rows
// may exist, a row lies by itself.
__host__ __device__ constexpr int part_rows(int R) { return R > 64 ? 32 : 1; }
// Where columns 4 c .. + 3 of row r of a slot lie.
__device__ __forceinline__ float* part_at(const AttnArgs& a, int slot, int r, int c) {
  const int n = part_rows(a.R), g = r / n;
  return a.part_o + ((size_t)slot * a.R + g * n) * a.d + ((size_t)c * n + (r - g * n)) * 4;
}

// One thread of every CTA: what its boundary's merge has to do (`any`: the CTA
// has tiles, `it` the item that holds its first).
__device__ __forceinline__ void note_shared(const AttnArgs& a, const Plan& pl, const Item& it, bool any) {
  Shared x;
  x.it = it;
  x.first = x.last = -1;
  const long long u0 = pl.Q * blockIdx.x;
  if (any && it.first < u0 && it.first >= u0 - pl.Q) {
    x.first = (int)blockIdx.x - 1;
    const long long rest = it.first + it.tiles - u0;  // tiles from the boundary on
    x.last = (int)blockIdx.x + (rest <= pl.Q ? 0 : (int)((unsigned)(rest - 1) / (unsigned)pl.Q));
  }
  a.shared[blockIdx.x] = x;
}

// Natural logarithm of the softmax's sum from its maximum (log2 domain) and scaled sum.
__device__ __forceinline__ float lse_of(float m, float l) {
  return l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

// What a row's sums of products are multiplied by: 1 / l.  A maximum passes over NaN, so that a row whose
// scores are NaN, or one of them infinite, has a NaN as its sum, and keeps it.  l = 0: zeros for a row
// that sees no key (of a tree: a node with no mask bit before an empty prefix), and NaN for one whose
// every score was -inf.
__device__ __forceinline__ float row_scale(const AttnArgs& a, int L, int tok, float l) {
  if (l != 0.f) return 1.f / l;
  bool sees = !a.w.N || L > 0;
#pragma unroll 1
  for (int w = 0; !sees && w < a.W; ++w) {
    const int n = a.w.N - 32 * w;
    sees = a.mask[(size_t)tok * a.W + w] & (n >= 32 ? 0xffffffffu : (1u << n) - 1u);
  }
  return sees ? __int_as_float(0x7fffffff) : 0.f;
}

// Tensor-core kernel (paged_attention_tc.cu): bf16, d <= 128 a multiple of 8,
// page_size a multiple of 8, at most 128 q heads per kv head.
medusa_status paged_attention_tc(const AttnArgs& a, cudaStream_t s);

}  // namespace paged
}  // namespace medusa
