// Logits of a verify pass as requests want them (penalties, biases, grammar masks), and the counts
// of tokens that the penalties go by.
//
// The mathematics is elementwise: z' of (row b, node n, token v) needs z, what is known of
// (b, v) (count, prompt bit, bias) and whether v lies on n's path or is masked.  All but the last two is
// z' = z f + s with f one of two factors, by z's sign, and s a sum, both of (b, v) alone: a thread works them
// out once for the tokens that it has and goes through the nodes with one multiply-add each.  The tokens
// on the paths, at most 17 a node and few of them among a block's, are sorted out into a list a node in
// shared memory with their results, which are written last.
//
// What bounds it: memory, z read and z' written once; it takes care that instructions do not (the first form took 30
// an element, of which 9 are left).  A thread has several loads of logits in flight, those of the next nodes while it
// writes the last ones'; where there are few nodes and no tree, of several places in a row.  The rows of all chunks of
// tokens, laid end to end, are divided evenly over the blocks that the SMs hold at once.  The paths are a warp's own
// work, beside the others': what it finds out takes four trips to memory one after the other, which all waited for
// when they shared it.  Measured: 16 trees of 57 nodes, 32000 tokens, bf16: 37.3 us, 4.8 TB/s (nothing asked for: 30.4
// us); one tree of 64, fp32: 6.7 us; 64 rows of bf16 logits, 50257 tokens: 10.4 us, 3.1 TB/s; 50258: 10.4; 32000: 5.4; 128256: 16.7.
#include <math.h>

#include <type_traits>

#include "common.cuh"
#include "host_util.h"

namespace medusa {
namespace logits {

constexpr int kThreads = 256;
constexpr int kBlocks = 4;               // that an SM holds at once
constexpr int kRowBlocks = 5;            // of few nodes
constexpr int kGroup = 32;               // nodes that a block takes together at most
constexpr int kPath = MEDUSA_MAX_DEPTH + 1;

struct Args {
  const void* z;
  long long ld;
  medusa_logits_rules r;
  const int32_t *tokens, *parent;  // parent NULL: no tree
  int B, N, V, W;                  // W: words of a bit row
  int chunks;                      // of a row's tokens
  uint32_t units;                  // rows of all chunks
  float* out;
  int in_place;
  int32_t* d_status;
};

// VEC logits as they lie in memory.
template <typename T, int VEC>
struct Raw {
  using Word = std::conditional_t<VEC == 1, T, std::conditional_t<sizeof(T) == 4, float4, uint2>>;
  Word w;
  __device__ __forceinline__ void load(const T* p) { w = *reinterpret_cast<const Word*>(p); }
  __device__ __forceinline__ float get(int i) const {
    if constexpr (VEC == 1) return load_elem(&w, 0);
    else if constexpr (sizeof(T) == 4) return i == 0 ? w.x : i == 1 ? w.y : i == 2 ? w.z : w.w;
    else return __uint_as_float(i == 0 ? w.x << 16 : i == 1 ? w.x & 0xffff0000u : i == 2 ? w.y << 16 : w.y & 0xffff0000u);
  }
};

// The mask row of a node, -1 for none.
__device__ __forceinline__ int mask_row_of(const Args& a, size_t row) {
  const int m = a.r.mask_row ? a.r.mask_row[row] : (int)row;
  if (m >= -1 && m < a.r.n_masks) return m;
  set_status(a.d_status, MEDUSA_DEV_BAD_INDEX);
  return -1;
}

// The result of a token on a node's path, which occurs there c times.  Counts may lie below zero, so that it may be unsaid
// all the same.  All that is asked for is on its way at once.
__device__ __forceinline__ float on_path(const Args& a, int b, size_t row, int v, int c, float x) {
  const int m = a.r.mask ? mask_row_of(a, row) : -1;
  const int before = a.r.counts ? a.r.counts[(size_t)b * a.V + v] : 0;
  const uint32_t prompt = a.r.prompt_bits ? a.r.prompt_bits[(size_t)b * a.W + (v >> 5)] >> (v & 31) : 0;
  const float rep = a.r.repetition ? a.r.repetition[b] : 1.f, fr = a.r.frequency ? a.r.frequency[b] : 0.f, pr = a.r.presence ? a.r.presence[b] : 0.f,
              e = a.r.bias ? a.r.bias[(a.r.bias_rows > 1 ? (size_t)b * a.V : 0) + v] : 0.f;
  if (m >= 0 && !((a.r.mask[(size_t)m * a.W + (v >> 5)] >> (v & 31)) & 1u)) return -INFINITY;
  c += before;
  if (c > 0 || (prompt & 1u)) x = x > 0.f ? x / rep : x * rep;
  return x - fr * (float)c - (c > 0 ? pr : 0.f) + e;
}

// All warps of a block, from places of their own.
__device__ __forceinline__ void block_sync() {
  __syncwarp();
  asm volatile("barrier.cta.sync.aligned 1, %0;" ::"n"(kThreads) : "memory");
}

// A thread has VEC neighbouring tokens, and NODES nodes at a time.  TREE: the last warp has the paths.
template <typename T, int VEC, int NODES, bool TREE>
__global__ void __launch_bounds__(kThreads, kBlocks) process_kernel(const __grid_constant__ Args a) {
  constexpr int MAIN = TREE ? kThreads - 32 : kThreads, WIDE = MAIN * VEC;  // threads with tokens, tokens of a chunk
  // The last warp's own.
  __shared__ int s_tok[TREE ? MEDUSA_MAX_NODES : 1], s_par[TREE ? MEDUSA_MAX_NODES : 1];
  __shared__ uint16_t s_col[TREE ? kGroup : 1][kPath];
  __shared__ float s_y[TREE ? kGroup : 1][kPath];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x;
  uint32_t u = (uint32_t)((uint64_t)a.units * blockIdx.x / gridDim.x);
  const uint32_t end = (uint32_t)((uint64_t)a.units * (blockIdx.x + 1) / gridDim.x);
#pragma unroll 1
  while (u < end) {
    // Nodes n0 .. n0 + nn - 1 of row b, one chunk of their tokens.
    const uint32_t item = u / (uint32_t)a.N;
    const int n0 = (int)(u - item * a.N), b = (int)(item / (uint32_t)a.chunks), v_lo = (int)(item - (uint32_t)b * a.chunks) * WIDE;
    const int nn = (int)min(TREE ? min((uint32_t)kGroup, end - u) : end - u, (uint32_t)(a.N - n0));
    const size_t row0 = (size_t)b * a.N + n0;
    u += nn;
    if (TREE && tid >= MAIN) {
      // A lane a node: its path's tokens in this chunk, then their results.
      const int lane = tid - MAIN;
      int listed = 0;
#pragma unroll 1
      for (int j = lane; j < n0 + nn; j += 32) {
        s_tok[j] = a.tokens[(size_t)b * a.N + j];
        s_par[j] = a.parent[j];
      }
      __syncwarp();
      if (lane < nn) {
        int j = n0 + lane;
#pragma unroll 1
        for (int steps = 0; j >= 0; ++steps) {
          const int t = s_tok[j], up = s_par[j];
          if (t < 0 || t >= a.V) {
            set_status(a.d_status, MEDUSA_DEV_BAD_INDEX);
          } else if (t >= v_lo && t < v_lo + WIDE) {
            s_col[lane][listed] = (uint16_t)(t - v_lo);
            s_y[lane][listed++] = load_elem(static_cast<const T*>(a.z), (row0 + lane) * a.ld + t);
          }
          if (j == 0 ? up != -1 : up < 0 || up >= j || steps == kPath - 1) {
            set_status(a.d_status, MEDUSA_DEV_BAD_TOPOLOGY);
            break;
          }
          j = up;
        }
      }
      if (a.in_place) block_sync();  // these logits are read before their places are written
#pragma unroll 1
      for (int k = 0; k < listed; ++k) {
        int c = 0;
#pragma unroll 1
        for (int h = 0; h < listed; ++h) c += s_col[lane][h] == s_col[lane][k];
        s_y[lane][k] = on_path(a, b, row0 + lane, v_lo + s_col[lane][k], c, s_y[lane][k]);
      }
      block_sync();  // the other results are written
#pragma unroll 1
      for (int k = 0; k < listed; ++k) a.out[(row0 + lane) * a.V + v_lo + s_col[lane][k]] = s_y[lane][k];
      __syncwarp();
      continue;
    }
    const int v0 = v_lo + tid * VEC, shift = v0 & 31;
    const bool in = v0 < a.V;
    int left = in ? nn : 0;  // nodes that this thread has still to write
    const T* zp = static_cast<const T*>(a.z) + row0 * a.ld + v0;
    float* yp = a.out + row0 * a.V + v0;
    const int32_t* rp = a.r.mask_row ? a.r.mask_row + row0 : nullptr;
    const uint32_t* mp = a.r.mask ? a.r.mask + (v0 >> 5) : nullptr;
    int next_row = (int)row0;  // where no rows of masks are named
    Raw<T, VEC> z[NODES];
    uint32_t allowed[NODES];
    int rows[NODES];
    // The next `n` nodes' logits; their mask rows; the masks of rows fetched before.
    auto fetch = [&](int n) {
#pragma unroll
      for (int j = 0; j < NODES; ++j, zp += a.ld)
        if (j < n) z[j].load(zp);
    };
    auto fetch_rows = [&](int n) {
      if (!mp) return;
#pragma unroll
      for (int j = 0; j < NODES; ++j) {
        rows[j] = -1;
        if (j < n) rows[j] = rp ? rp[j] : next_row + j;
      }
      if (rp) rp += NODES;
      next_row += NODES;
    };
    auto fetch_masks = [&] {
#pragma unroll
      for (int j = 0; j < NODES; ++j) {
        allowed[j] = 0xffffffffu;
        if (mp) {
          if (rows[j] < -1 || rows[j] >= a.r.n_masks) {
            set_status(a.d_status, MEDUSA_DEV_BAD_INDEX);
          } else if (rows[j] >= 0) {
            allowed[j] = mp[(size_t)rows[j] * a.W] >> shift;
          }
        }
      }
    };
    fetch_rows(left);
    fetch(left);
    // Factors for z > 0 and otherwise, and what is added.
    float pos[VEC], neg[VEC], add[VEC];
    {
      int c[VEC];
      const uint32_t prompt = in && a.r.prompt_bits ? a.r.prompt_bits[(size_t)b * a.W + (v0 >> 5)] >> shift : 0;
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        c[i] = in && a.r.counts ? a.r.counts[(size_t)b * a.V + v0 + i] : 0;
        add[i] = in && a.r.bias ? a.r.bias[(a.r.bias_rows > 1 ? (size_t)b * a.V : 0) + v0 + i] : 0.f;
      }
      const float rep = a.r.repetition ? a.r.repetition[b] : 1.f, inv = 1.f / rep, fr = a.r.frequency ? a.r.frequency[b] : 0.f,
                  pr = a.r.presence ? a.r.presence[b] : 0.f;
      fetch_masks();
      fetch_rows(left - NODES);
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const bool said = c[i] > 0 || ((prompt >> i) & 1u);
        pos[i] = said ? inv : 1.f;
        neg[i] = said ? rep : 1.f;
        if (c[i] != 0) add[i] -= fmaf(fr, (float)c[i], c[i] > 0 ? pr : 0.f);
      }
    }
    if (TREE && a.in_place) block_sync();
    auto write = [&](const Raw<T, VEC>& x, uint32_t may) {
      float y[VEC];
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const float e = x.get(i);
        y[i] = may & (1u << i) ? fmaf(e, e > 0.f ? pos[i] : neg[i], add[i]) : -INFINITY;
      }
      if constexpr (VEC == 4) *reinterpret_cast<float4*>(yp) = make_float4(y[0], y[1], y[2], y[3]);
      else *yp = y[0];
      yp += a.V;
    };
#pragma unroll 1
    for (; left > 0; left -= NODES) {
      Raw<T, VEC> now[NODES];
      uint32_t may[NODES];
#pragma unroll
      for (int j = 0; j < NODES; ++j) {
        now[j] = z[j];
        may[j] = allowed[j];
      }
      if (left >= 2 * NODES) {
        fetch(NODES);
        fetch_masks();
        fetch_rows(left - 2 * NODES);
      } else if (left > NODES) {
        fetch(left - NODES);
        fetch_masks();
      }
      if (left >= NODES) {
#pragma unroll
        for (int j = 0; j < NODES; ++j) write(now[j], may[j]);
      } else {
#pragma unroll
        for (int j = 0; j < NODES; ++j)
          if (j < left) write(now[j], may[j]);
      }
    }
    if (TREE) block_sync();
  }
}

// Few nodes and no tree: a thread has COLS times VEC tokens of a row, and nothing is worked out for other rows.  Seven places
// of one token and kRowBlocks come from a sweep at 64 rows of 50257 tokens alone.
template <typename T, int VEC, int COLS>
__global__ void __launch_bounds__(kThreads, kRowBlocks) rows_kernel(const __grid_constant__ Args a) {
  constexpr int STEP = kThreads * VEC, WIDE = STEP * COLS;
  pdl_wait();
  pdl_trigger();
  uint32_t u = (uint32_t)((uint64_t)a.units * blockIdx.x / gridDim.x);
  const uint32_t end = (uint32_t)((uint64_t)a.units * (blockIdx.x + 1) / gridDim.x);
#pragma unroll 1
  for (; u < end; ++u) {
    const uint32_t row = u / (uint32_t)a.chunks;
    const int v_lo = (int)(u - row * a.chunks) * WIDE, v0 = v_lo + threadIdx.x * VEC, shift = v0 & 31, b = (int)(row / (uint32_t)a.N);
    const bool whole = v_lo + WIDE <= a.V;
    const int m = a.r.mask ? mask_row_of(a, row) : -1;
    const float rep = a.r.repetition ? a.r.repetition[b] : 1.f, fr = a.r.frequency ? a.r.frequency[b] : 0.f, pr = a.r.presence ? a.r.presence[b] : 0.f;
    const T* zp = static_cast<const T*>(a.z) + (size_t)row * a.ld + v0;
    const int32_t* cp = a.r.counts ? a.r.counts + (size_t)b * a.V + v0 : nullptr;
    const float* ep = a.r.bias ? a.r.bias + (a.r.bias_rows > 1 ? (size_t)b * a.V : 0) + v0 : nullptr;
    const uint32_t* pp = a.r.prompt_bits ? a.r.prompt_bits + (size_t)b * a.W + (v0 >> 5) : nullptr;
    float* yp = a.out + (size_t)row * a.V + v0;
    auto chunk = [&](auto here) {  // here(q): place q is inside the row
      Raw<T, VEC> z[COLS];
      int c[COLS][VEC];
      float e[COLS][VEC];
      uint32_t prompt[COLS], allowed[COLS];
#pragma unroll
      for (int q = 0; q < COLS; ++q)
        if (here(q)) z[q].load(zp + q * STEP);
#pragma unroll
      for (int q = 0; q < COLS; ++q)
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          c[q][i] = cp && here(q) ? cp[q * STEP + i] : 0;
          e[q][i] = ep && here(q) ? ep[q * STEP + i] : 0.f;
        }
#pragma unroll
      for (int q = 0; q < COLS; ++q) prompt[q] = pp && here(q) ? pp[q * (STEP / 32)] >> shift : 0;
      const uint32_t* mp = a.r.mask + (m >= 0 ? (size_t)m * a.W + (v0 >> 5) : 0);
#pragma unroll
      for (int q = 0; q < COLS; ++q) allowed[q] = m >= 0 && here(q) ? mp[q * (STEP / 32)] >> shift : 0xffffffffu;
      const float inv = 1.f / rep;
      int signs = 0;
#pragma unroll
      for (int q = 0; q < COLS; ++q)
#pragma unroll
        for (int i = 0; i < VEC; ++i) signs |= c[q][i];
      auto write = [&](auto below) {  // whether counts below zero are among them: their part is a branch of its own
#pragma unroll
        for (int q = 0; q < COLS; ++q) {
          float y[VEC];
#pragma unroll
          for (int i = 0; i < VEC; ++i) {
            const float x = z[q].get(i), f = c[q][i] > 0 || (prompt[q] & (1u << i)) ? (x > 0.f ? inv : rep) : 1.f;
            float s = c[q][i] > 0 ? e[q][i] - (fr * (float)c[q][i] + pr) : e[q][i];
            if (below()) s -= fr * (float)min(c[q][i], 0);
            y[i] = allowed[q] & (1u << i) ? fmaf(x, f, s) : -INFINITY;
          }
          if (here(q)) {
            if constexpr (VEC == 4) *reinterpret_cast<float4*>(yp + q * STEP) = make_float4(y[0], y[1], y[2], y[3]);
            else yp[q * STEP] = y[0];
          }
        }
      };
      if (signs >= 0) write(std::false_type());
      else write(std::true_type());
    };
    if (whole) chunk([](int) { return true; });
    else chunk([&](int q) { return v0 + q * STEP < a.V; });
  }
}

// ------------------------------------------------------------------ counts

// Grid (ceil(S / 256), B).  Sums of whole numbers, so that the order of the atomic additions changes nothing.  Bound by the
// launch (7 prompts of up to 4099 tokens: 1.7 us in a row, 2.8 as calls of their own).
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

// A warp a row: lane i has node i of the path.  Bound by the launch and three trips to memory (1.2 us in a row, 2.7 as
// calls of their own).
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

template <typename T, int VEC>
static void launch(Args a, cudaStream_t s) {
  constexpr int NODES = VEC == 4 ? (sizeof(T) == 4 ? 2 : 4) : 6, COLS = VEC == 4 ? (sizeof(T) == 4 ? 1 : 2) : 7;
  const bool few = !a.parent && a.N < 4;
  const long long wide = few ? kThreads * VEC * COLS : (a.parent ? kThreads - 32 : kThreads) * VEC, most = (long long)(few ? kRowBlocks : kBlocks) * device_sm_count();
  a.chunks = (int)((a.V + wide - 1) / wide);
  a.units = (uint32_t)((long long)a.N * a.B * a.chunks);
  const dim3 grid((unsigned)(a.units < most ? a.units : most));
  if (few) launch_pdl(rows_kernel<T, VEC, COLS>, grid, dim3(kThreads), 0, s, a);
  else if (a.parent) launch_pdl(process_kernel<T, VEC, NODES, true>, grid, dim3(kThreads), 0, s, a);
  else launch_pdl(process_kernel<T, VEC, NODES, false>, grid, dim3(kThreads), 0, s, a);
}

}  // namespace logits
}  // namespace medusa

using namespace medusa;
using namespace medusa::logits;

static bool at4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
// Sizes whose last block's columns or threads, and a step of 65535 behind them, stay inside int32.
static bool fits(int n) { return n >= 1 && n < 0x7fffffff - 65535; }

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
  a.in_place = in_place;
  a.d_status = d_status;
  if (rows * ((V + kThreads - 33) / (kThreads - 32)) > 0xffffffffll) return MEDUSA_ERR_INVALID_ARG;  // more than a GPU holds
  const bool vec = V % 4 == 0 && ld % 4 == 0 && ((uintptr_t)logits & (4 * es - 1)) == 0 && aligned16(out);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (dt == MEDUSA_F32) vec ? launch<float, 4>(a, s) : launch<float, 1>(a, s);
  else vec ? launch<uint16_t, 4>(a, s) : launch<uint16_t, 1>(a, s);
  return launch_status();
}

extern "C" medusa_status medusa_count_tokens(const int32_t* tokens, int B, int S, int V, int32_t* counts, uint32_t* prompt_bits,
                                             int32_t* d_status, medusa_stream_t stream) {
  if (!fits(B) || S < 0 || (S > 0 && !fits(S)) || !fits(V) || (!counts && !prompt_bits) || (S > 0 && !tokens)) return MEDUSA_ERR_INVALID_ARG;
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
