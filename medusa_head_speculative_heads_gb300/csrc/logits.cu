// Logits of a verify pass as requests want them (penalties, biases, grammar masks), and the counts
// of tokens that the penalties go by.
//
// The mathematics is elementwise: z' of (row b, node n, token v) needs z, what is known of
// (b, v) (count, prompt bit, bias) and whether v lies on n's path or is masked.  What bounds it:
// memory, z read and z' written once.  So a thread owns VEC neighbouring tokens of one row b, loads what is
// known of them once and goes through the nodes, kNodes logit loads in flight at a time; the tokens on
// the paths, at most 17 a node and hardly ever in a block's columns, are sorted out beforehand into a
// list a node in shared memory.
#include <math.h>

#include "common.cuh"
#include "host_util.h"

namespace medusa {
namespace logits {

constexpr int kThreads = 256;
constexpr int kGroup = 32;               // nodes of a block at most
constexpr int kPath = MEDUSA_MAX_DEPTH + 1;

struct Args {
  const void* z;
  long long ld;
  medusa_logits_rules r;
  const int32_t *tokens, *parent;  // parent NULL: no tree
  int B, N, V, W;                  // W: words of a bit row
  int chunks, groups, group;       // column chunks, groups of nodes, nodes of a group
  float* out;
  int32_t* d_status;
};

template <typename T, int VEC>
__device__ __forceinline__ void load_z(const T* p, float* z) {
  if constexpr (VEC == 1) {
    z[0] = load_elem(p, 0);
  } else if constexpr (sizeof(T) == 4) {
    const float4 v = *reinterpret_cast<const float4*>(p);
    z[0] = v.x; z[1] = v.y; z[2] = v.z; z[3] = v.w;
  } else {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    z[0] = __uint_as_float(v.x << 16); z[1] = __uint_as_float(v.x & 0xffff0000u);
    z[2] = __uint_as_float(v.y << 16); z[3] = __uint_as_float(v.y & 0xffff0000u);
  }
}

// Grid (chunks * groups, B).
template <typename T, int VEC, int NODES>
__global__ void __launch_bounds__(kThreads) process_kernel(const __grid_constant__ Args a) {
  __shared__ int s_tok[MEDUSA_MAX_NODES], s_par[MEDUSA_MAX_NODES];
  __shared__ int s_row[kGroup];            // mask row of a node, -1: none
  __shared__ int s_n[kGroup];              // tokens of its path in this block's columns
  __shared__ uint16_t s_col[kGroup][kPath];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, chunk = blockIdx.x % a.chunks, grp = blockIdx.x / a.chunks;
  const int n0 = grp * a.group, nn = min(a.group, a.N - n0);
  const int v_lo = chunk * (kThreads * VEC), v0 = v_lo + tid * VEC;
  const bool in = v0 < a.V;
  for (int b = blockIdx.y; b < a.B; b += gridDim.y) {
    const size_t row0 = (size_t)b * a.N + n0;
    // The nodes' tokens on their way to the root that fall into the block's columns.
    if (a.parent)
      for (int j = tid; j < n0 + nn; j += kThreads) {
        s_tok[j] = a.tokens[(size_t)b * a.N + j];
        s_par[j] = a.parent[j];
      }
    if (tid < nn) {
      int m = -1;
      if (a.r.mask) {
        const long long x = a.r.mask_row ? a.r.mask_row[row0 + tid] : (long long)(row0 + tid);
        if (x >= 0 && x < a.r.n_masks) m = (int)x;
        else if (x != -1) set_status(a.d_status, MEDUSA_DEV_BAD_INDEX);
      }
      s_row[tid] = m;
      s_n[tid] = 0;
    }
    __syncthreads();
    if (a.parent && tid < nn) {
      int k = 0, j = n0 + tid;
      for (int steps = 0; j >= 0; ++steps) {
        const int t = s_tok[j], up = s_par[j];
        if (t < 0 || t >= a.V) set_status(a.d_status, MEDUSA_DEV_BAD_INDEX);
        else if (t >= v_lo && t < v_lo + kThreads * VEC) s_col[tid][k++] = (uint16_t)(t - v_lo);
        if (j == 0 ? up != -1 : up < 0 || up >= j || steps == kPath - 1) {
          set_status(a.d_status, MEDUSA_DEV_BAD_TOPOLOGY);
          break;
        }
        j = up;
      }
      s_n[tid] = k;
    }
    // What is known of this thread's tokens.
    int cnt[VEC];
    float bias[VEC];
    uint32_t said = 0;  // bit i: in the prompt
    const float rep = a.r.repetition ? a.r.repetition[b] : 1.f, fr = a.r.frequency ? a.r.frequency[b] : 0.f,
                pr = a.r.presence ? a.r.presence[b] : 0.f;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      cnt[i] = 0;
      bias[i] = 0.f;
    }
    if (in) {
      if (a.r.counts)
#pragma unroll
        for (int i = 0; i < VEC; ++i) cnt[i] = a.r.counts[(size_t)b * a.V + v0 + i];
      if (a.r.bias)
#pragma unroll
        for (int i = 0; i < VEC; ++i) bias[i] = a.r.bias[(a.r.bias_rows > 1 ? (size_t)b * a.V : 0) + v0 + i];
      if (a.r.prompt_bits) said = a.r.prompt_bits[(size_t)b * a.W + (v0 >> 5)] >> (v0 & 31);
    }
    __syncthreads();
    for (int j0 = 0; j0 < nn; j0 += NODES) {
      float z[NODES][VEC];
      uint32_t allowed[NODES];
#pragma unroll
      for (int j = 0; j < NODES; ++j) {
        allowed[j] = 0xffffffffu;
        if (in && j0 + j < nn) {
          load_z<T, VEC>(static_cast<const T*>(a.z) + (row0 + j0 + j) * a.ld + v0, z[j]);
          const int m = s_row[j0 + j];
          if (m >= 0) allowed[j] = a.r.mask[(size_t)m * a.W + (v0 >> 5)] >> (v0 & 31);
        }
      }
#pragma unroll
      for (int j = 0; j < NODES; ++j) {
        if (j0 + j >= nn || !in) break;
        int c[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) c[i] = cnt[i];
        for (int k = 0; k < s_n[j0 + j]; ++k) {
          const int col = s_col[j0 + j][k] - tid * VEC;
#pragma unroll
          for (int i = 0; i < VEC; ++i) c[i] += col == i;
        }
        float y[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          float x = z[j][i];
          if (c[i] > 0 || ((said >> i) & 1u)) x = x > 0.f ? x / rep : x * rep;
          if (c[i] > 0) x = x - fr * (float)c[i] - pr;
          y[i] = (allowed[j] >> i) & 1u ? x + bias[i] : -INFINITY;
        }
        float* dst = a.out + (row0 + j0 + j) * a.V + v0;
        if constexpr (VEC == 4) *reinterpret_cast<float4*>(dst) = make_float4(y[0], y[1], y[2], y[3]);
        else dst[0] = y[0];
      }
    }
    __syncthreads();  // the lists are read
  }
}

// ------------------------------------------------------------------ counts

// Grid (ceil(S / 256), B).
__global__ void __launch_bounds__(256)
count_tokens_kernel(const int32_t* tokens, int B, int S, int V, int32_t* counts, uint32_t* bits, int32_t* d_status) {
  pdl_wait();
  pdl_trigger();
  const int s = blockIdx.x * 256 + threadIdx.x, W = (V + 31) / 32;
  if (s >= S) return;
  for (int b = blockIdx.y; b < B; b += gridDim.y) {
    const int t = tokens[(size_t)b * S + s];
    if (t >= V) set_status(d_status, MEDUSA_DEV_BAD_INDEX);
    if (t < 0 || t >= V) continue;
    if (counts) atomicAdd(counts + (size_t)b * V + t, 1);
    if (bits) atomicOr(bits + (size_t)b * W + (t >> 5), 1u << (t & 31));
  }
}

// A warp a row: lane i has node i of the path.
__global__ void __launch_bounds__(128)
count_accepted_kernel(const int32_t* tokens, const int32_t* path_nodes, const int32_t* accept_len, int B, int N, int D1, int V,
                      int32_t* counts, int32_t* d_status) {
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (b >= B) return;
  const int n = accept_len[b], node = lane < D1 ? path_nodes[(size_t)b * D1 + lane] : -1;
  const bool mine = lane < n;
  const int t = mine && node >= 0 && node < N ? tokens[(size_t)b * N + node] : -1;
  const bool bad = n < 1 || n > D1 || (mine && (t < 0 || t >= V));
  if (__any_sync(0xffffffffu, bad)) {
    if (lane == 0) set_status(d_status, MEDUSA_DEV_BAD_INDEX);
    return;
  }
  if (mine) atomicAdd(counts + (size_t)b * V + t, 1);
}

template <typename T, int VEC, int NODES>
static void launch(const Args& a, int rows, cudaStream_t s) {
  launch_pdl(process_kernel<T, VEC, NODES>, dim3((unsigned)(a.chunks * a.groups), rows), dim3(kThreads), 0, s, a);
}

}  // namespace logits
}  // namespace medusa

using namespace medusa;
using namespace medusa::logits;

static bool at4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
// Sizes whose last block's columns or threads stay inside int32.
static bool fits(int n) { return n >= 1 && n < 0x7fffffff - 65536; }

extern "C" medusa_status medusa_logits_process(const void* logits, int64_t ld, medusa_dtype dt, const medusa_logits_rules* rules,
                                               const int32_t* tokens, const medusa_dev_topology* t, int B, int N, int V, float* out,
                                               int32_t* d_status, medusa_stream_t stream) {
  if (!logits || !rules || !out || !dtype_ok(dt) || B < 1 || N < 1 || !fits(V) || ld < V) return MEDUSA_ERR_INVALID_ARG;
  const medusa_logits_rules& r = *rules;
  if (t && (!tokens || !t->parent || t->n_nodes != N || N > MEDUSA_MAX_NODES)) return MEDUSA_ERR_INVALID_ARG;
  const long long rows = (long long)B * N;
  if (rows > 0x7fffffffll || ld > (1ll << 40)) return MEDUSA_ERR_INVALID_ARG;
  if (r.bias && r.bias_rows != 1 && r.bias_rows != B) return MEDUSA_ERR_INVALID_ARG;
  if (r.mask && (r.n_masks < 1 || (!r.mask_row && r.n_masks != rows))) return MEDUSA_ERR_INVALID_ARG;
  const size_t es = dtype_bytes(dt);
  const uintptr_t ints = (uintptr_t)out | (uintptr_t)r.counts | (uintptr_t)r.prompt_bits | (uintptr_t)r.repetition | (uintptr_t)r.frequency |
                         (uintptr_t)r.presence | (uintptr_t)r.bias | (uintptr_t)r.mask | (uintptr_t)r.mask_row | (uintptr_t)d_status |
                         (t ? (uintptr_t)tokens | (uintptr_t)t->parent : 0);
  if ((ints & 3) || ((uintptr_t)logits & (es - 1))) return MEDUSA_ERR_INVALID_ARG;
  Args a{};
  a.W = (V + 31) / 32;
  const size_t nz = ((size_t)(rows - 1) * ld + V) * es, no = (size_t)rows * V * 4, nb = (size_t)B * 4, bits = (size_t)a.W * 4;
  const bool in_place = logits == out && dt == MEDUSA_F32 && ld == V;
  if (overlaps_any({out, no}, {{in_place ? nullptr : logits, nz}, {r.counts, nb * V}, {r.prompt_bits, B * bits}, {r.repetition, nb},
                               {r.frequency, nb}, {r.presence, nb}, {r.bias, r.bias ? (size_t)r.bias_rows * V * 4 : 0},
                               {r.mask, r.mask ? r.n_masks * bits : 0}, {r.mask ? r.mask_row : nullptr, (size_t)rows * 4},
                               {t ? tokens : nullptr, (size_t)rows * 4}, {t ? t->parent : nullptr, (size_t)N * 4}, {d_status, 4}}))
    return MEDUSA_ERR_ALIAS;
  a.z = logits;
  a.ld = ld;
  a.r = r;
  a.tokens = tokens;
  a.parent = t ? t->parent : nullptr;
  a.B = B;
  a.N = N;
  a.V = V;
  a.out = out;
  a.d_status = d_status;
  const bool vec = V % 4 == 0 && ld % 4 == 0 && ((uintptr_t)logits & (4 * es - 1)) == 0 && aligned16(out);
  const int cols = kThreads * (vec ? 4 : 1);
  a.chunks = (V + cols - 1) / cols;
  a.group = N < 8 ? N : 8;
  a.groups = (N + a.group - 1) / a.group;
  if ((long long)a.chunks * a.groups > 0x7fffffffll) return MEDUSA_ERR_INVALID_ARG;
  const int gy = B < 65535 ? B : 65535;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (dt == MEDUSA_F32) vec ? launch<float, 4, 4>(a, gy, s) : launch<float, 1, 8>(a, gy, s);
  else vec ? launch<uint16_t, 4, 4>(a, gy, s) : launch<uint16_t, 1, 8>(a, gy, s);
  return launch_status();
}

extern "C" medusa_status medusa_count_tokens(const int32_t* tokens, int B, int S, int V, int32_t* counts, uint32_t* prompt_bits,
                                             int32_t* d_status, medusa_stream_t stream) {
  if (B < 1 || S < 0 || (S > 0 && !fits(S)) || !fits(V) || (!counts && !prompt_bits) || (S > 0 && !tokens)) return MEDUSA_ERR_INVALID_ARG;
  if (!at4(tokens) || !at4(counts) || !at4(prompt_bits) || !at4(d_status)) return MEDUSA_ERR_INVALID_ARG;
  const size_t nt = (size_t)B * S * 4, nc = (size_t)B * V * 4, nb = (size_t)B * ((V + 31) / 32) * 4;
  if (overlaps_any({counts, nc}, {{tokens, nt}, {prompt_bits, nb}, {d_status, 4}}) || overlaps_any({prompt_bits, nb}, {{tokens, nt}, {d_status, 4}}))
    return MEDUSA_ERR_ALIAS;
  if (S == 0) return MEDUSA_OK;
  launch_pdl(count_tokens_kernel, dim3((S + 255) / 256, B < 65535 ? B : 65535), dim3(256), 0, reinterpret_cast<cudaStream_t>(stream), tokens, B, S,
             V, counts, prompt_bits, d_status);
  return launch_status();
}

extern "C" medusa_status medusa_count_accepted(const int32_t* tokens, const int32_t* path_nodes, const int32_t* accept_len, int B, int N,
                                               int Dmax, int V, int32_t* counts, int32_t* d_status, medusa_stream_t stream) {
  if (!tokens || !path_nodes || !accept_len || !counts || !fits(B) || N < 1 || N > MEDUSA_MAX_NODES || Dmax < 0 || Dmax > MEDUSA_MAX_DEPTH || !fits(V))
    return MEDUSA_ERR_INVALID_ARG;
  if (!at4(tokens) || !at4(path_nodes) || !at4(accept_len) || !at4(counts) || !at4(d_status)) return MEDUSA_ERR_INVALID_ARG;
  const size_t nb = (size_t)B * 4;
  if (overlaps_any({counts, nb * V}, {{tokens, nb * N}, {path_nodes, nb * (Dmax + 1)}, {accept_len, nb}, {d_status, 4}})) return MEDUSA_ERR_ALIAS;
  launch_pdl(count_accepted_kernel, dim3((B + 3) / 4), dim3(128), 0, reinterpret_cast<cudaStream_t>(stream), tokens, path_nodes, accept_len, B, N,
             Dmax + 1, V, counts, d_status);
  return launch_status();
}
