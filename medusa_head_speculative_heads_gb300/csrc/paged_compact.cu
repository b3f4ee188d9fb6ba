// medusa_paged_compact: the accepted path's tree keys and values enter the
// paged cache.
//
// Skill-pack guide ("Medusa 多解码头推理加速全解析"), section "树形验证": the
// accepted tokens' keys and values join past_key_values; here the rows lie in
// the pages page_table names.
//
// Latency bounds the call (a path is a few rows of Hkv x d elements in each
// layer).  One CTA moves one (layer, sequence, path slot, K or V) row at a
// time; its threads check the whole path and its pages side by side, so a
// sequence that cannot be entered whole writes nothing.  new_len is written by
// the first threads of the grid, or by a second kernel when it shares memory
// with prefix_len, which every CTA of the first one reads.
#include <limits.h>

#include "host_util.h"
#include "paged.cuh"

namespace medusa {
namespace paged {

struct CompactArgs {
  void *k_pages, *v_pages;
  const void *kt, *vt;
  const int32_t *path_nodes, *accept_len, *prefix_len;
  int32_t *new_len, *d_status;
  Cache cache;
  int nl, B, N, D1;  // D1: path slots
  int words;         // per row of Hkv x d elements
  int rows;          // nl * B * D1 * 2
};

// Why sequence b cannot be entered (MEDUSA_DEV_OK: it can), from its lengths alone.
__device__ __forceinline__ int length_error(const CompactArgs& a, int b, int& L, int& A) {
  L = a.prefix_len[b];
  A = a.accept_len[b];
  if (L < 0) return MEDUSA_DEV_BAD_LENGTH;
  if (A < 1 || A > a.D1) return MEDUSA_DEV_BAD_INDEX;
  return L > a.cache.rows() - A ? MEDUSA_DEV_CACHE_OVERFLOW : MEDUSA_DEV_OK;
}
__device__ __forceinline__ bool slot_ok(const CompactArgs& a, int b, int L, int j) {
  const int n = a.path_nodes[(size_t)b * a.D1 + j];
  return n >= 0 && n < a.N && pool_row(a.cache, b, L + j) >= 0;
}

__device__ __forceinline__ int new_len_of(const CompactArgs& a, int b) {
  int L, A;
  bool ok = length_error(a, b, L, A) == MEDUSA_DEV_OK;
  for (int j = 0; ok && j < A; ++j) ok = slot_ok(a, b, L, j);
  return ok ? L + A : L;
}

template <typename WORD>
__global__ void __launch_bounds__(256) paged_compact_kernel(const __grid_constant__ CompactArgs a, int write_len) {
  pdl_wait();
  pdl_trigger();
  if (write_len) {
    const long long b = blockIdx.x * (long long)blockDim.x + threadIdx.x;
    if (b < a.B) a.new_len[b] = new_len_of(a, (int)b);
  }
  for (unsigned row = blockIdx.x; row < (unsigned)a.rows; row += gridDim.x) {  // a sum past 2^31 is no row
    int r = (int)row;
    const int kv = r & 1;
    r >>= 1;
    const int i = r % a.D1;
    r /= a.D1;
    const int b = r % a.B, l = r / a.B;
    int L, A;
    int err = length_error(a, b, L, A);
    if (!err && i >= A) continue;
    if (!err) {
      const int j = threadIdx.x;
      if (__syncthreads_or(j < A && !slot_ok(a, b, L, j))) err = MEDUSA_DEV_BAD_INDEX;
    }
    if (err) {
      if (l == 0 && i == 0 && kv == 0 && threadIdx.x == 0) set_status(a.d_status, err);
      continue;
    }
    const int node = a.path_nodes[(size_t)b * a.D1 + i];
    const WORD* from = static_cast<const WORD*>(kv ? a.vt : a.kt) + (((size_t)l * a.B + b) * a.N + node) * a.words;
    const size_t to_row = (size_t)l * a.cache.n_pages * a.cache.page_size + pool_row(a.cache, b, L + i);
    WORD* to = static_cast<WORD*>(kv ? a.v_pages : a.k_pages) + to_row * a.words;
    int w = threadIdx.x;
    for (; w + (int)blockDim.x < a.words; w += 2 * blockDim.x) {
      const WORD x = from[w], y = from[w + blockDim.x];
      to[w] = x;
      to[w + blockDim.x] = y;
    }
    if (w < a.words) to[w] = from[w];
  }
}

__global__ void paged_len_kernel(const __grid_constant__ CompactArgs a) {
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.x * blockDim.x + threadIdx.x;
  if (b < a.B) a.new_len[b] = new_len_of(a, b);
}

}  // namespace paged
}  // namespace medusa

using namespace medusa;
using namespace medusa::paged;

extern "C" medusa_status medusa_paged_compact(void* k_pages, void* v_pages, const int32_t* page_table, const void* kt,
                                              const void* vt, const int32_t* path_nodes, const int32_t* accept_len,
                                              const int32_t* prefix_len, int32_t* new_len, int n_layers, int B, int N,
                                              int Hkv, int d, int n_pages, int page_size, int max_pages, int Dmax,
                                              medusa_dtype dt, int32_t* d_status, medusa_stream_t stream) {
  if (!k_pages || !v_pages || !page_table || !kt || !vt || !path_nodes || !accept_len || !prefix_len || !new_len)
    return MEDUSA_ERR_INVALID_ARG;
  if (n_layers < 1 || B < 1 || N < 1 || N > MEDUSA_MAX_NODES || Hkv < 1 || Hkv > 65535 || d < 1 || d > MEDUSA_MAX_HEAD_DIM)
    return MEDUSA_ERR_INVALID_ARG;
  if (Dmax < 0 || Dmax > MEDUSA_MAX_DEPTH || !dtype_ok(dt) || !cache_sizes_ok(n_layers, B, n_pages, page_size, max_pages))
    return MEDUSA_ERR_INVALID_ARG;
  const long long rows = (long long)n_layers * B * (Dmax + 1) * 2;
  if (rows > INT_MAX) return MEDUSA_ERR_INVALID_ARG;
  const size_t es = dtype_bytes(dt), row_bytes = (size_t)Hkv * d * es;
  const uintptr_t all = (uintptr_t)k_pages | (uintptr_t)v_pages | (uintptr_t)kt | (uintptr_t)vt;
  const uintptr_t ints = (uintptr_t)page_table | (uintptr_t)path_nodes | (uintptr_t)accept_len | (uintptr_t)prefix_len |
                         (uintptr_t)new_len | (uintptr_t)d_status;
  if ((all & (es - 1)) || (ints & 3)) return MEDUSA_ERR_INVALID_ARG;
  const size_t np = (size_t)n_layers * n_pages * page_size * row_bytes, nt = (size_t)n_layers * B * N * row_bytes;
  if (overlaps(k_pages, np, v_pages, np)) return MEDUSA_ERR_ALIAS;
  for (const void* pool : {(const void*)k_pages, (const void*)v_pages})
    if (overlaps(pool, np, kt, nt) || overlaps(pool, np, vt, nt)) return MEDUSA_ERR_ALIAS;
  const size_t nb = (size_t)B * 4;
  if (overlaps_any({new_len, nb}, {{k_pages, np}, {v_pages, np}, {kt, nt}, {vt, nt}})) return MEDUSA_ERR_ALIAS;
  for (const Region& r : {Region{page_table, nb * max_pages}, Region{path_nodes, nb * (Dmax + 1)}, Region{accept_len, nb}, Region{prefix_len, nb}})
    if (overlaps_any(r, {{k_pages, np}, {v_pages, np}})) return MEDUSA_ERR_ALIAS;
  if (overlaps(new_len, nb, accept_len, nb) || overlaps(new_len, nb, path_nodes, nb * (Dmax + 1)) ||
      overlaps(new_len, nb, page_table, nb * max_pages) || (new_len != prefix_len && overlaps(new_len, nb, prefix_len, nb)))
    return MEDUSA_ERR_ALIAS;
  const int wb = row_bytes % 16 == 0 && (all & 15) == 0 ? 16 : row_bytes % 4 == 0 && (all & 3) == 0 ? 4 : 2;
  CompactArgs a{};
  a.k_pages = k_pages;
  a.v_pages = v_pages;
  a.kt = kt;
  a.vt = vt;
  a.path_nodes = path_nodes;
  a.accept_len = accept_len;
  a.prefix_len = prefix_len;
  a.new_len = new_len;
  a.d_status = d_status;
  a.cache = Cache{page_table, n_pages, page_size, max_pages};
  a.nl = n_layers;
  a.B = B;
  a.N = N;
  a.D1 = Dmax + 1;
  a.words = (int)(row_bytes / wb);
  a.rows = (int)rows;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int threads = a.words >= 256 ? 256 : (a.words + 31) / 32 * 32;  // at least one warp: D1 <= 17 slots to check
  long long blocks = rows, cap = (long long)device_sm_count() * 16;
  if (blocks > cap) blocks = cap;
  if (blocks * threads < B) blocks = (B + threads - 1) / threads;
  const int own_len = new_len != prefix_len ? 1 : 0;
  if (wb == 16) launch_pdl(paged_compact_kernel<uint4>, dim3((unsigned)blocks), dim3(threads), 0, s, a, own_len);
  else if (wb == 4) launch_pdl(paged_compact_kernel<uint32_t>, dim3((unsigned)blocks), dim3(threads), 0, s, a, own_len);
  else launch_pdl(paged_compact_kernel<uint16_t>, dim3((unsigned)blocks), dim3(threads), 0, s, a, own_len);
  if (!own_len) launch_pdl(paged_len_kernel, dim3((B + 127) / 128), dim3(128), 0, s, a);
  return launch_status();
}
