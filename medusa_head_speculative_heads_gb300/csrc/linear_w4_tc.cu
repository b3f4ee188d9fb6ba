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

constexpr int kThreads = 512;              // W, products, x, -; 2 x 4 unpacking; 4 reading out
constexpr int kRows = 256;                 // features of a tile
constexpr int kCols = 128;                 // columns of a block
constexpr int kMaxTN = 192;
constexpr int kSlotsW = 4;
constexpr int kMaxSlotsX = 16;
constexpr uint32_t kSlotW = kRows * kCols / 2;
constexpr uint32_t kHalfW = kSlotW / 2;
constexpr uint32_t kRing = 229376;         // 224 KB for both rings
constexpr uint32_t kTmemCols = 512;
constexpr int kMinBlocks = 2;              // of a CTA
constexpr int kPolls = 1 << 23;            // of a wait that does not sleep: some 100 ns each
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
  uint64_t a_full[2][4], a_empty[2][4], d_full[2], d_empty[2], drain;
  uint32_t tmem;
  volatile int abort;
  int w_loads, x_loads;
};
constexpr uint32_t kSmem = kRing + sizeof(Tail);
static_assert(kSmem <= 232448, "shared memory of a CTA");

__host__ __device__ __forceinline__ long long work_begin(long long work, int grid, int c) { return work * c / grid; }
__device__ __forceinline__ int work_owner(long long work, int grid, long long w) { return (int)(((w + 1) * grid - 1) / work); }

// A CTA's blocks, one after the other.
struct Walk {
  int tile, kb, left;
};
__device__ __forceinline__ Walk walk_of(const Tc& p) {
  const long long w0 = work_begin(p.work, p.grid, blockIdx.x), w1 = work_begin(p.work, p.grid, blockIdx.x + 1);
  const int tile = (int)(w0 / p.kblocks);
  return {tile, (int)(w0 - (long long)tile * p.kblocks), (int)(w1 - w0)};
}
__device__ __forceinline__ void step(const Tc& p, Walk& x) {
  --x.left;
  if (++x.kb == p.kblocks) {
    x.kb = 0;
    ++x.tile;
  }
}
// Blocks of the tile the walk is in that are this CTA's.
__device__ __forceinline__ int tile_blocks(const Tc& p, const Walk& x) { return min(x.left, p.kblocks - x.kb); }

__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(ok));
  return ok != 0;
}
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
  const bool ok = mbar_wait_bounded(bar, parity, abort, kWaitNs);
  return __all_sync(0xffffffffu, ok);
}
__device__ __forceinline__ bool test_wait(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile("{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
               : "=r"(ok)
               : "r"(smem_u32(bar)), "r"(parity)
               : "memory");
  return ok != 0;
}
// Every lane with `need` waits for a phase of a barrier of its own, all at once.
__device__ __forceinline__ bool lanes_wait(uint64_t* bar, uint32_t parity, bool need, volatile int* abort) {
  bool ok = !need;
#pragma unroll 1
  for (int n = kPolls; n > 0; --n) {
    if (!ok) ok = test_wait(bar, parity);
    if (__all_sync(0xffffffffu, ok)) {
      __syncwarp();
      return true;
    }
    if ((n & 15) == 0 && __any_sync(0xffffffffu, *abort)) return false;
  }
  *abort = 1;
  return false;
}
__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// The scales and zeros of a thread's row in a block of columns: GROUPS of them.
template <int GROUPS>
struct Raw {
  uint16_t s[GROUPS];
  uint8_t z[GROUPS];
};
template <int GROUPS>
__device__ __forceinline__ Raw<GROUPS> load_groups(const Tc& p, const Walk& x, int row) {
  Raw<GROUPS> r;
  const int n = min(x.tile / p.ntiles * kRows + row, p.a.Nout - 1);
  const int g0 = x.kb * GROUPS, ng = p.a.K >> p.a.glog;
#pragma unroll
  for (int i = 0; i < GROUPS; ++i) {
    r.s[i] = 0;  // behind the last column: weights of 0
    r.z[i] = 8;
    if (g0 + i < ng) {
      const size_t at = (size_t)(g0 + i) * p.a.Nout + n;
      r.s[i] = p.a.scales[at];
      if (p.a.zeros) r.z[i] = p.a.zeros[at];
    }
  }
  return r;
}

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
      mbar_init(&tail->w_empty[i], 8);
    }
    for (int i = 0; i < p.NX; ++i) {
      mbar_init(&tail->x_full[i], 1);
      mbar_init(&tail->x_empty[i], 1);
    }
    for (int h = 0; h < 2; ++h) {
      for (int i = 0; i < 4; ++i) {
        mbar_init(&tail->a_full[h][i], 4);
        mbar_init(&tail->a_empty[h][i], 1);
      }
      mbar_init(&tail->d_full[h], 1);
      mbar_init(&tail->d_empty[h], 4);
    }
    mbar_init(&tail->drain, 1);
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
    int i = 0;
    for (; x.left > 0; step(p, x), ++i) {
      const int s = i % kSlotsW;
      if (i >= kSlotsW && !warp_wait(&tail->w_empty[s], (uint32_t)(i / kSlotsW - 1) & 1u, abort)) break;
      if (elect_one()) {
        mbar_expect_tx(&tail->w_full[s], kSlotW);
        for (int h = 0; h < 2; ++h)
          tma_load_2d(smem + s * kSlotW + h * kHalfW, &tm_w, &tail->w_full[s], x.kb * (kCols / 2), x.tile / p.ntiles * kRows + h * 128);
      }
      __syncwarp();
    }
    if (lane == 0) tail->w_loads = i;
  } else if (warp == 2) {
    // ------------------------------------------------------------ tokens
    int j = 0;
    bool alive = true;
    for (; x.left > 0 && alive; step(p, x)) {
      for (int u = 0; u < 2; ++u, ++j) {
        const int s = j % p.NX;
        if (j >= p.NX && !(alive = warp_wait(&tail->x_empty[s], (uint32_t)(j / p.NX - 1) & 1u, abort))) break;
        if (elect_one()) {
          mbar_expect_tx(&tail->x_full[s], (uint32_t)p.TN * 128);
          if (!(p.withhold && j == 0))
            tma_load_2d(ring_x + s * (p.TN * 128), &tm_x, &tail->x_full[s], x.kb * kCols + u * 64, x.tile % p.ntiles * p.TN);
        }
        __syncwarp();
      }
    }
    if (lane == 0) tail->x_loads = j;
  } else if (warp == 1) {
    // ------------------------------------------------------------ products
    const uint32_t idesc = idesc_bf16_f32(128, p.TN, false, false);
    const uint32_t a0 = tmem + 2 * p.DN;
    int j = 0, seg = 0;
    bool alive = true;
    while (x.left > 0 && alive) {
      const int nb = tile_blocks(p, x);
      for (int k = 0; k < 2 * nb && alive; ++k, ++j) {
        const int sx = j % p.NX, b = j & (p.NA - 1);
        const uint32_t px = (uint32_t)(j / p.NX) & 1u, pa = (uint32_t)(j / p.NA) & 1u;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint64_t* bar = lane == 0 ? &tail->a_full[h][b] : lane == 1 ? &tail->x_full[sx] : &tail->d_empty[h];
          const bool need = lane == 0 || (lane == 1 && h == 0) || (lane == 2 && k == 0 && seg > 0);
          if (!(alive = lanes_wait(bar, lane == 0 ? pa : lane == 1 ? px : (uint32_t)(seg - 1) & 1u, need, abort))) break;
          tc_fence_after();
          if (elect_one()) {
            const uint64_t xd = smem_desc_sw128(smem_u32(ring_x + sx * (p.TN * 128)), 16, 1024);
            const uint32_t at = a0 + (h * p.NA + b) * 32;
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) mma_bf16_ts(tmem + h * p.DN, at + 8 * kk, xd + 2 * kk, idesc, k > 0 || kk > 0);
            mma_commit(&tail->a_empty[h][b]);
            if (h == 1) mma_commit(&tail->x_empty[sx]);
            if (k == 2 * nb - 1) mma_commit(&tail->d_full[h]);
          }
          __syncwarp();
        }
      }
      ++seg;
      x.left -= nb;
      x.kb = 0;
      ++x.tile;
    }
    if (elect_one()) {
      // This warp's products and the arrivals they signal, before tensor and shared memory go away.
      mma_commit(&tail->drain);
      mbar_wait_bounded(&tail->drain, 0, nullptr, kDrainNs);
    }
    __syncwarp();
  } else if (warp >= 4 && warp < 12) {
    // ------------------------------------------------------------ unpacking: half h, rows 32 q4 ..
    const int h = (warp - 4) >> 2, q4 = warp & 3, row = 32 * q4 + lane;
    const uint32_t a0 = tmem + ((uint32_t)(32 * q4) << 16) + 2 * p.DN + h * p.NA * 32;
    Walk ahead = x;
    int i = 0;
    bool alive = true;
    // Scales two blocks ahead: they take a round trip to memory.
    auto next = [&] {
      Raw<GROUPS> r{};
      if (ahead.left > 0) {
        r = load_groups<GROUPS>(p, ahead, h * 128 + row);
        step(p, ahead);
      }
      return r;
    };
    auto block = [&](Raw<GROUPS>& raw) {
      Group g[GROUPS];
#pragma unroll
      for (int k = 0; k < GROUPS; ++k) g[k] = group_of(raw.s[k], raw.z[k]);
      raw = next();
      const int s = i % kSlotsW;
      if (!warp_wait(&tail->w_full[s], (uint32_t)(i / kSlotsW) & 1u, abort)) return false;
      const uint8_t* w = smem + s * kSlotW + h * kHalfW + row * 64;
      uint4 v[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) v[c] = *reinterpret_cast<const uint4*>(w + 16 * (c ^ ((row >> 1) & 3)));  // 64-byte swizzle
      warp_arrive(&tail->w_empty[s]);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int j = 2 * i + u, b = j & (p.NA - 1);
        uint32_t r[32];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const uint4& t = v[2 * u + c];
          const Group& gr = g[(2 * u + c) * GROUPS / 4];
          unpack(t.x, gr, r + 16 * c);
          unpack(t.y, gr, r + 16 * c + 4);
          unpack(t.z, gr, r + 16 * c + 8);
          unpack(t.w, gr, r + 16 * c + 12);
        }
        if (j >= p.NA && !warp_wait(&tail->a_empty[h][b], (uint32_t)(j / p.NA - 1) & 1u, abort)) return false;
        tc_fence_after();
        tmem_st32u(a0 + 32 * b, r);
        tmem_wait_st();
        tc_fence_before();
        warp_arrive(&tail->a_full[h][b]);
      }
      ++i;
      return true;
    };
    Raw<GROUPS> r0 = next(), r1 = next();
    const int n = x.left;
    while (i < n && alive) {
      alive = block(r0);
      if (alive && i < n) alive = block(r1);
    }
  } else if (warp >= 12) {
    // ------------------------------------------------------------ reading out
    const int q4 = warp & 3, m = 32 * q4 + lane, first = x.tile;
    const uint32_t lanes = tmem + ((uint32_t)(32 * q4) << 16);
    int seg = 0;
    bool alive = true;
    for (; x.left > 0 && alive; ++seg) {
      const int nb = tile_blocks(p, x);
      const bool whole = nb == p.kblocks;
      const int t0 = x.tile % p.ntiles * p.TN, f0 = x.tile / p.ntiles * kRows;
      float* part = p.part + ((size_t)blockIdx.x * 2 + (x.tile == first ? 0 : 1)) * p.TN * kRows;
      for (int h = 0; h < 2; ++h) {
        if (!(alive = warp_wait(&tail->d_full[h], seg & 1, abort))) break;
        tc_fence_after();
        const int n = f0 + h * 128 + m;
#pragma unroll 1
        for (int c = 0; c < p.TN; c += 32) {
          float v[32];
          __syncwarp();
          tmem_ld32(lanes + h * p.DN + c, v);
          tmem_wait_ld();
          if (whole) {
            if (n < p.a.Nout) {
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (t0 + c + e < p.a.T && c + e < p.TN) store_y(p.a, t0 + c + e, n, v[e]);
            }
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (c + e < p.TN) part[(size_t)(c + e) * kRows + h * 128 + m] = v[e];
          }
        }
        tc_fence_before();
        warp_arrive(&tail->d_empty[h]);
      }
      x.left -= nb;
      x.kb = 0;
      ++x.tile;
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
  p.NA = 2 * p.DN + 2 * 4 * 32 <= (int)kTmemCols ? 4 : 2;
  p.NX = (int)((kRing - kSlotsW * kSlotW) / (p.TN * 128));
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
