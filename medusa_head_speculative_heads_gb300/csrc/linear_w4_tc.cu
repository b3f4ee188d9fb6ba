// medusa_linear_w4 on tcgen05 tensor cores: many tokens.
//
// y^T = W x^T in tiles of 256 features by up to 192 tokens.  Weights come as they are kept, 64 bytes a
// row and 128 columns, by TMA; eight warps unpack them into tensor memory, where the matrix instruction reads its
// first operand (a thread has a row and 64 columns of it: 32 words, four loads of 16 bytes from
// shared memory), so that unpacked weights never pass through shared memory.  The tokens are the second
// operand, by TMA in slots of 64 columns.  256 features share a tile of tokens: with weights this
// small it is the tokens whose traffic counts.
//
// The two halves of 128 features have a sum in tensor memory, buffers of unpacked weights and
// four unpacking warps of their own; one warp issues their products in turn, so that a half's sum is read out
// under the other's products.
//
// The blocks of 128 columns of all tiles, laid end to end (the token tiles of a feature tile
// behind one another), are divided evenly over the CTAs, one an SM.  A tile that several CTAs share
// leaves a partial sum each, at most two a CTA, which a second kernel adds in the CTAs' order.
//
// Every wait is bounded: a timeout sets MEDUSA_DEV_TIMEOUT, all roles stop, copies and products in
// flight are waited for and tensor memory is freed.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <math.h>

#include "host_util.h"
#include "linear_w4.h"
#include "sm100.cuh"

namespace medusa {
namespace w4 {
using namespace sm100;

constexpr int kThreads = 768;              // W, products, x, products; 4 x 4 unpacking; 4 reading out
constexpr int kUnpackers = 16;
constexpr int kRows = 256;                 // features of a tile
constexpr int kCols = 128;                 // columns of a block
constexpr int kMaxTN = 192;
constexpr int kSlotsW = 4;
constexpr int kMaxSlotsX = 8;
constexpr uint32_t kSlotW = kRows * kCols / 2;
constexpr uint32_t kHalfW = kSlotW / 2;
constexpr uint32_t kRing = 229376;         // 224 KB for both rings
constexpr uint32_t kTmemCols = 512;
constexpr int kMinBlocks = 2;              // of a CTA
constexpr uint64_t kWaitNs = 1000000000ull;
constexpr uint64_t kDrainNs = 100000000ull;

struct Tc {
  Args a;
  int TN, DN, NA, NX;  // tokens of a tile, columns of a sum, buffers of unpacked weights and slots of tokens
  int ntiles, kblocks, grid;
  long long work;
  float* part;         // [grid][2][TN][256]
  int withhold;        // failure test: the first tokens are never loaded
};

struct Tail {
  uint64_t w_full[kSlotsW], w_empty[kSlotsW], x_full[kMaxSlotsX], x_empty[kMaxSlotsX];
  uint64_t a_full[2][2], a_empty[2][2], d_full[2], d_empty[2], drain[2];
  uint32_t tmem;
  volatile int abort;
  int w_loads, x_loads;
};
constexpr uint32_t kSmem = kRing + sizeof(Tail);
static_assert(kSmem <= 232448, "shared memory of a CTA");

__host__ __device__ __forceinline__ long long work_begin(long long work, int grid, int c) { return work * c / grid; }
__device__ __forceinline__ int work_owner(long long work, int grid, long long w) { return (int)(((w + 1) * grid - 1) / work); }

// A CTA's blocks, one after the other: feature tile, token tile, block of columns.
struct Walk {
  int mt, nt, kb, left;
};
__device__ __forceinline__ Walk walk_of(const Tc& p) {
  const long long w0 = work_begin(p.work, p.grid, blockIdx.x), w1 = work_begin(p.work, p.grid, blockIdx.x + 1);
  const int tile = (int)(w0 / p.kblocks), mt = tile / p.ntiles;
  return {mt, tile - mt * p.ntiles, (int)(w0 - (long long)tile * p.kblocks), (int)(w1 - w0)};
}
__device__ __forceinline__ void next_tile(const Tc& p, Walk& x) {
  x.kb = 0;
  if (++x.nt == p.ntiles) {
    x.nt = 0;
    ++x.mt;
  }
}
__device__ __forceinline__ void step(const Tc& p, Walk& x) {
  --x.left;
  if (++x.kb == p.kblocks) next_tile(p, x);
}
// Blocks of the tile the walk is in that are this CTA's.
__device__ __forceinline__ int tile_blocks(const Tc& p, const Walk& x) { return min(x.left, p.kblocks - x.kb); }

// A place in a ring and the parity of its present round.
struct Ring {
  int i = 0;
  uint32_t round = 0;
  __device__ __forceinline__ void next(int n) {
    if (++i == n) {
      i = 0;
      ++round;
    }
  }
  // The phase that ends when this place is full; the one that ended when it was last emptied.
  __device__ __forceinline__ uint32_t full() const { return round & 1u; }
  __device__ __forceinline__ uint32_t empty() const { return (round - 1u) & 1u; }
  __device__ __forceinline__ bool used() const { return round > 0; }
};

__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(ok));
  return ok != 0;
}
// Barriers by their shared-memory addresses: what a wait costs in instructions, the unpacking warps have less for
// their work.
__device__ __forceinline__ bool try_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile("{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
               : "=r"(ok)
               : "r"(bar), "r"(parity)
               : "memory");
  return ok != 0;
}
// What follows a try that came back empty, out of line: the roles' loops have to stay in the instruction caches next
// to one another.
__device__ __noinline__ bool wait_longer(uint32_t bar, uint32_t parity, volatile int* abort) {
  const uint64_t t0 = global_timer_ns();
  while (!try_wait(bar, parity)) {
    if (*abort) return false;
    if ((int64_t)(global_timer_ns() - t0) > (int64_t)kWaitNs) {
      *abort = 1;
      return false;
    }
  }
  return true;
}
// All lanes wait for a phase; true when all saw it end.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort) {
  if (__all_sync(0xffffffffu, try_wait(bar, parity))) return true;
  const bool ok = wait_longer(bar, parity, abort);
  return __all_sync(0xffffffffu, ok);
}
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort) { return warp_wait(smem_u32(bar), parity, abort); }
// A value that is the same in all lanes, known to be so by the compiler.
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __shfl_sync(0xffffffffu, v, 0); }
// Descriptors of K-major operands with 128-byte swizzle are a constant half and an address in units of 16 bytes.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint64_t desc_of(uint32_t lo) { return ((uint64_t)kDescHi << 32) | lo; }
__device__ __forceinline__ void warp_arrive(uint32_t bar, int lane) {
  __syncwarp();
  if (lane == 0) asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// The scales and zeros of a row in a block of columns: GROUPS of them.
template <int GROUPS>
struct Raw {
  uint32_t s[GROUPS], z[GROUPS];
};
// Those of the blocks a thread unpacks, which are two apart.
template <int GROUPS>
struct Scales {
  Walk x;
  int row;
  size_t at, two;  // of the block; from it to the next but one of the same tile
  __device__ __forceinline__ void start(const Tc& p) {
    at = (size_t)(x.kb * GROUPS) * p.a.Nout + min(x.mt * kRows + row, p.a.Nout - 1);
  }
  __device__ __forceinline__ Scales(const Tc& p, const Walk& w, int r) : x(w), row(r), two((size_t)(2 * GROUPS) * p.a.Nout) { start(p); }
  __device__ __forceinline__ void next(const Tc& p) {
    x.left -= 2;
    x.kb += 2;
    at += two;
    if (x.kb >= p.kblocks) {
      x.kb -= 2;
      x.left += 2;
      step(p, x);
      step(p, x);
      start(p);
    }
  }
  __device__ __forceinline__ Raw<GROUPS> load(const Tc& p) const {
    Raw<GROUPS> r;
#pragma unroll
    for (int i = 0; i < GROUPS; ++i) {
      r.s[i] = 0;  // behind the last column: weights of 0
      r.z[i] = 8;
      if (x.left > 0 && (GROUPS == 1 || x.kb * kCols + kCols / GROUPS * i < p.a.K)) {
        r.s[i] = p.a.scales[at + (size_t)i * p.a.Nout];
        if (p.a.zeros) r.z[i] = p.a.zeros[at + (size_t)i * p.a.Nout];
      }
    }
    return r;
  }
};

template <int GROUPS>
__global__ void __launch_bounds__(kThreads, 1)
tc_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ Tc p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  Tail* tail = reinterpret_cast<Tail*>(smem + kRing);
  volatile int* abort = &tail->abort;
  if (smem_u32(smem) & 1023u) {  // the same in every thread
    if (threadIdx.x == 0) set_status(p.a.d_status, MEDUSA_DEV_TIMEOUT);
    return;
  }
  uint8_t* ring_x = smem + kSlotsW * kSlotW;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    tail->abort = 0;
    for (int i = 0; i < kSlotsW; ++i) {
      mbar_init(&tail->w_full[i], 1);
      mbar_init(&tail->w_empty[i], kUnpackers / 2);
    }
    for (int i = 0; i < p.NX; ++i) {
      mbar_init(&tail->x_full[i], 1);
      mbar_init(&tail->x_empty[i], 2);
    }
    for (int h = 0; h < 2; ++h) {
      for (int i = 0; i < 2; ++i) {
        mbar_init(&tail->a_full[h][i], 4);
        mbar_init(&tail->a_empty[h][i], 1);
      }
      mbar_init(&tail->d_full[h], 1);
      mbar_init(&tail->drain[h], 1);
      mbar_init(&tail->d_empty[h], 4);
    }
    fence_mbar_init();
  }
  if (warp == 1) {
    __syncwarp();
    tmem_alloc(&tail->tmem, kTmemCols);
    tmem_relinquish();
  }
  Walk x = walk_of(p);
  if (warp == 0 && lane == 0) {
    tma_prefetch(&tm_w);
    tma_prefetch(&tm_x);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_wait();
  pdl_trigger();
  const uint32_t tmem = tail->tmem;

  if (warp == 0) {
    // ------------------------------------------------------------ weights as they are kept
    int n = 0;
    for (Ring w; x.left > 0; step(p, x), w.next(kSlotsW), ++n) {
      if (w.used() && !warp_wait(&tail->w_empty[w.i], w.empty(), abort)) break;
      if (elect_one()) {
        mbar_expect_tx(&tail->w_full[w.i], kSlotW);
        for (int h = 0; h < 2; ++h)
          tma_load_2d(smem + w.i * kSlotW + h * kHalfW, &tm_w, &tail->w_full[w.i], x.kb * (kCols / 2), x.mt * kRows + h * 128);
      }
      __syncwarp();
    }
    if (lane == 0) tail->w_loads = n;
  } else if (warp == 2) {
    // ------------------------------------------------------------ tokens
    int n = 0;
    for (Ring t; x.left > 0; step(p, x), t.next(p.NX), ++n) {
      if (t.used() && !warp_wait(&tail->x_empty[t.i], t.empty(), abort)) break;
      if (elect_one()) {
        mbar_expect_tx(&tail->x_full[t.i], (uint32_t)p.TN * 256);
        for (int u = 0; u < 2; ++u)
          if (!(p.withhold && n == 0 && u == 0))
            tma_load_2d(ring_x + (2 * t.i + u) * (p.TN * 128), &tm_x, &tail->x_full[t.i], x.kb * kCols + u * 64, x.nt * p.TN);
      }
      __syncwarp();
    }
    if (lane == 0) tail->x_loads = n;
  } else if (warp == 1 || warp == 3) {
    // ------------------------------------------------------------ products of half h
    // Issued by an elected lane of the whole warp, their addresses known to be the same in all lanes: by a lane on
    // its own a product took 80 clocks to issue, so 11.
    const int h = warp >> 1;
    const uint32_t idesc = uniform(idesc_bf16_f32(128, p.TN, false, false)), d = uniform(tmem + h * p.DN),
                   a0 = uniform(tmem + 2 * p.DN + h * p.NA * 64), x0 = (smem_u32(ring_x) >> 4) | (1u << 16), half = uniform(p.TN * 8);
    Ring t;
    uint32_t i = 0;  // blocks
    bool alive = true;
    for (int seg = 0; x.left > 0 && alive; ++seg) {
      const int nb = tile_blocks(p, x);
#pragma unroll 1
      for (int k = 0; k < nb; ++k, ++i) {
        const uint32_t xd = uniform(x0 + t.i * p.TN * 16), a = uniform(a0 + (i & (p.NA - 1)) * 64);
        if (k == 0 && seg > 0 && !(alive = warp_wait(&tail->d_empty[h], (uint32_t)(seg - 1) & 1u, abort))) break;
        if (!(alive = warp_wait(&tail->x_full[t.i], t.full(), abort) && warp_wait(&tail->a_full[h][i & 1], (i >> 1) & 1u, abort))) break;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            mma_bf16_ts(d, a + 8 * kk, desc_of(xd + (kk >> 2) * half + 2 * (kk & 3)), idesc, kk > 0 || k > 0);
          mma_commit(&tail->a_empty[h][i & 1]);
          mma_commit(&tail->x_empty[t.i]);
          if (k == nb - 1) mma_commit(&tail->d_full[h]);
        }
        __syncwarp();
        t.next(p.NX);
      }
      x.left -= nb;
      next_tile(p, x);
    }
    if (elect_one()) {
      // This warp's products and the arrivals they signal, before tensor and shared memory go away.
      mma_commit(&tail->drain[h]);
      mbar_wait_bounded(&tail->drain[h], 0, nullptr, kDrainNs);
    }
    __syncwarp();
  } else if (warp >= 4 && warp < 4 + kUnpackers) {
    // ------------------------------------------------------------ unpacking: half h, every second block, rows 32 q4 ..
    // A set has the blocks of one parity, and so the same slots of the ring and the same barriers each time: it
    // passes over no phase of them.
    const int h = (warp >> 2) & 1, set = warp >= 4 + kUnpackers / 2, q4 = warp & 3, row = 32 * q4 + lane;
    const uint32_t to = tmem + ((uint32_t)(32 * q4) << 16) + 2 * p.DN + (h * p.NA + (set & (p.NA - 1))) * 64;
    const uint32_t sw = 16 * ((row >> 1) & 3);  // 64-byte swizzle
    // The buffer is free once the products of the block before it there are done: of two blocks ago, or,
    // with one buffer, of the other set's.
    const uint32_t free = smem_u32(&tail->a_empty[h][p.NA == 2 ? set : set ^ 1]), filled = smem_u32(&tail->a_full[h][set]);
    uint32_t free_phase = 1, slot = set;
    bool first = p.NA == 2 || set == 0;  // nothing was there before
    uint32_t round = 0;
    if (set) step(p, x);
    Scales<GROUPS> scales(p, x, h * 128 + row);
    Raw<GROUPS> raw = scales.load(p);
#pragma unroll 1
    for (int left = x.left; left > 0; left -= 2) {
      Group g[GROUPS];
#pragma unroll
      for (int k = 0; k < GROUPS; ++k) g[k] = group_of(raw.s[k], raw.z[k]);
      scales.next(p);
      raw = scales.load(p);  // of the set's next block: they take a round trip to memory
      if (!warp_wait(smem_u32(&tail->w_full[0]) + 8 * slot, round, abort)) break;
      const uint32_t w = smem_u32(smem) + slot * kSlotW + h * kHalfW + row * 64;
      uint4 v[4];
#pragma unroll
      for (int c = 0; c < 4; ++c)
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v[c].x), "=r"(v[c].y), "=r"(v[c].z), "=r"(v[c].w) : "r"(w + ((16 * c) ^ sw)) : "memory");
      uint32_t r[32];
      auto half_block = [&](int u) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const Group& gr = g[(2 * u + c) * GROUPS / 4];
          unpack(v[2 * u + c].x, gr, r + 16 * c);
          unpack(v[2 * u + c].y, gr, r + 16 * c + 4);
          unpack(v[2 * u + c].z, gr, r + 16 * c + 8);
          unpack(v[2 * u + c].w, gr, r + 16 * c + 12);
        }
      };
      half_block(0);
      warp_arrive(smem_u32(&tail->w_empty[0]) + 8 * slot, lane);
      slot ^= 2;
      round ^= slot < 2;
      if (first) first = false;
      else if (!warp_wait(free, free_phase ^= 1, abort)) break;
      tc_fence_after();
      tmem_st32u(to, r);
      half_block(1);
      __syncwarp();
      tmem_st32u(to + 32, r);
      tmem_wait_st();
      tc_fence_before();
      warp_arrive(filled, lane);
    }
  } else if (warp >= 4 + kUnpackers) {
    // ------------------------------------------------------------ reading out
    const int q4 = warp & 3, m = 32 * q4 + lane;
    const uint32_t lanes = tmem + ((uint32_t)(32 * q4) << 16);
    bool alive = true;
    for (int seg = 0; x.left > 0 && alive; ++seg) {
      const int nb = tile_blocks(p, x);
      const bool whole = nb == p.kblocks;
      const int t0 = x.nt * p.TN, tokens = min(p.TN, p.a.T - t0);
      for (int h = 0; h < 2; ++h) {
        if (!(alive = warp_wait(&tail->d_full[h], seg & 1, abort))) break;
        tc_fence_after();
        const int n = x.mt * kRows + h * 128 + m;
        float* part = p.part + ((size_t)blockIdx.x * 2 + (seg ? 1 : 0)) * p.TN * kRows + h * 128 + m;
        size_t at = (size_t)t0 * p.a.Nout + n;
#pragma unroll 1
        for (int c = 0; c < p.TN; c += 16, part += 16 * kRows) {
          float v[16];
          __syncwarp();
          tmem_ld16(lanes + h * p.DN + c, v);
          tmem_wait_ld();
          if (!whole) {
#pragma unroll
            for (int e = 0; e < 16; ++e) part[e * kRows] = v[e];
          } else if (n < p.a.Nout) {
            const int more = tokens - c;
            if (p.a.y32) {
              float* y = static_cast<float*>(p.a.y);
#pragma unroll
              for (int e = 0; e < 16; ++e, at += p.a.Nout)
                if (e < more) y[at] = v[e];
            } else {
              uint16_t* y = static_cast<uint16_t*>(p.a.y);
#pragma unroll
              for (int e = 0; e < 16; ++e, at += p.a.Nout)
                if (e < more) y[at] = bf16_rn(v[e]);
            }
          }
        }
        tc_fence_before();
        warp_arrive(smem_u32(&tail->d_empty[h]), lane);
      }
      x.left -= nb;
      next_tile(p, x);
    }
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (threadIdx.x == 0 && *abort) {
    set_status(p.a.d_status, MEDUSA_DEV_TIMEOUT);
    // No copy may land after exit: wait (bounded) for the last phase of every load.
    for (int i = max(0, tail->w_loads - kSlotsW); i < tail->w_loads; ++i)
      mbar_wait_bounded(&tail->w_full[i % kSlotsW], (uint32_t)(i / kSlotsW) & 1u, nullptr, kDrainNs);
    for (int j = max(0, tail->x_loads - p.NX); j < tail->x_loads; ++j)
      mbar_wait_bounded(&tail->x_full[j % p.NX], (uint32_t)(j / p.NX) & 1u, nullptr, kDrainNs);
  }
  if (warp == 1) {
    __syncwarp();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// The partial sums of shared tiles, in the CTAs' order.  Block x looks at the boundary in front of CTA x + 1:
// when it lies inside a tile and no earlier boundary does, the block adds that tile's parts: a
// thread has 4 features, blockIdx.y and the thread's row choose the tokens.
__global__ void __launch_bounds__(256) tc_reduce_kernel(const __grid_constant__ Tc p) {
  pdl_wait();
  pdl_trigger();
  const int c = blockIdx.x + 1;
  const long long wc = work_begin(p.work, p.grid, c), wp = work_begin(p.work, p.grid, c - 1);
  if (wc % p.kblocks == 0) return;
  const int tile = (int)(wc / p.kblocks);
  const long long base = (long long)tile * p.kblocks;
  if (wp > base) return;
  const int last = work_owner(p.work, p.grid, base + p.kblocks - 1);
  const int row = (threadIdx.x & 63) * 4, n = tile / p.ntiles * kRows + row, t0 = tile % p.ntiles * p.TN;
  if (n >= p.a.Nout) return;
  const size_t slot = (size_t)p.TN * kRows;
  const float* first = p.part + ((size_t)(c - 1) * 2 + (wp == base ? 0 : 1)) * slot;  // the tile is that CTA's first or its last
  for (int col = blockIdx.y * 4 + (threadIdx.x >> 6); col < p.TN; col += gridDim.y * 4) {
    if (t0 + col >= p.a.T) break;
    const size_t off = (size_t)col * kRows + row;
    float4 s = __ldcg(reinterpret_cast<const float4*>(first + off));
    for (int k = c; k <= last; ++k) {
      const float4 v = __ldcg(reinterpret_cast<const float4*>(p.part + (size_t)k * 2 * slot + off));
      s.x += v.x;
      s.y += v.y;
      s.z += v.z;
      s.w += v.w;
    }
    const float v[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n + i < p.a.Nout) store_y(p.a, t0 + col, n + i, v[i]);
  }
}

// ------------------------------------------------------------------ host side

static PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    cudaGetLastError();
    return static_cast<PFN_cuTensorMapEncodeTiled_v12000>(nullptr);
  }();
  return fn;
}

// [rows][cols] with `pitch` bytes between rows, boxes of bc columns by br rows.
static bool make_map(CUtensorMap* m, CUtensorMapDataType ty, const void* base, long long cols, long long rows, long long pitch, int bc, int br,
                     CUtensorMapSwizzle sw) {
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)pitch};
  const cuuint32_t box[2] = {(cuuint32_t)bc, (cuuint32_t)br}, es[2] = {1, 1};
  return encode_fn()(m, ty, 2, const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, sw,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The division of the work: shared by the workspace query and the call.
static Tc plan(int T, int K, int Nout) {
  Tc p{};
  p.ntiles = (T + kMaxTN - 1) / kMaxTN;
  p.TN = ((T + p.ntiles - 1) / p.ntiles + 15) / 16 * 16;
  p.ntiles = (T + p.TN - 1) / p.TN;
  p.DN = (p.TN + 31) / 32 * 32;
  p.NA = 2 * p.DN + 2 * 2 * 64 <= (int)kTmemCols ? 2 : 1;
  p.NX = (int)((kRing - kSlotsW * kSlotW) / (p.TN * 256));
  if (p.NX > kMaxSlotsX) p.NX = kMaxSlotsX;
  p.kblocks = (K + kCols - 1) / kCols;
  p.work = (long long)((Nout + kRows - 1) / kRows) * p.ntiles * p.kblocks;
  long long g = p.work / kMinBlocks;
  if (g > device_sm_count()) g = device_sm_count();
  p.grid = g < 1 ? 1 : (int)g;
  return p;
}
static bool shared_tiles(const Tc& p) {
  for (int c = 1; c < p.grid; ++c)
    if (work_begin(p.work, p.grid, c) % p.kblocks != 0) return true;
  return false;
}

size_t tc_workspace(int T, int K, int Nout) {
  const Tc p = plan(T, K, Nout);
  return shared_tiles(p) ? (size_t)p.grid * 2 * p.TN * kRows * sizeof(float) : 0;
}

medusa_status tc_launch(const Args& a, float* part, int withhold, cudaStream_t s) {
  if (!encode_fn()) return MEDUSA_ERR_CUDA;
  Tc p = plan(a.T, a.K, a.Nout);
  p.a = a;
  p.part = part;
  p.withhold = withhold;
  CUtensorMap mw, mx;
  if (!make_map(&mw, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.q, a.K / 2, a.Nout, a.K / 2, kCols / 2, 128, CU_TENSOR_MAP_SWIZZLE_64B) ||
      !make_map(&mx, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.x, a.K, a.T, a.ldx * 2, 64, p.TN, CU_TENSOR_MAP_SWIZZLE_128B))
    return MEDUSA_ERR_CUDA;
  auto kern = a.glog == 5 ? tc_kernel<4> : a.glog == 6 ? tc_kernel<2> : tc_kernel<1>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem) != cudaSuccess) return MEDUSA_ERR_CUDA;
  launch_pdl(kern, dim3(p.grid), dim3(kThreads), kSmem, s, mw, mx, p);
  if (shared_tiles(p)) launch_pdl(tc_reduce_kernel, dim3(p.grid - 1, (p.TN + 15) / 16), dim3(256), 0, s, p);
  return launch_status();
}

}  // namespace w4
}  // namespace medusa
