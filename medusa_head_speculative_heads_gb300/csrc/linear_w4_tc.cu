// medusa_linear_w4 on tcgen05 tensor cores: many tokens.
//
// y^T = W x^T in tiles of up to 256 features by up to 128 tokens.  Weights come as they are kept, 64 bytes a
// row and 128 columns, by TMA; sixteen warps unpack them into tensor memory, where the matrix instruction reads its
// first operand (a thread has a row's 128 columns: 16 words, four loads of 16 bytes from shared memory), so that
// unpacked weights never pass through shared memory.  The tokens are the second operand, by TMA.  The features
// share a tile of tokens: with weights this small it is the tokens whose traffic counts.
//
// The two halves of a tile's features, up to 128 each, have a sum and buffers of unpacked weights in tensor memory, a
// warp that issues their products and two sets of four unpacking warps, which take blocks of 128 columns in turn.
//
// The work is divided into equal tiles: their height is chosen so that they fill the SMs in whole rounds (a CTA takes
// one after the other, without a pause in the rings).  Where there are too few of them, the CTAs of a
// cluster share a tile's columns: each sums up its blocks, sends the other CTAs their tokens' sums through
// distributed shared memory, and adds what it receives in the CTAs' order.
//
// What bounds it: for prompts the tensor cores and the power they take (2311 tokens, 11008 features of 4096 columns: 134 to
// 148 us by the machine, 1550 to 1410 TFLOP/s, tensor pipe 80 %); for a few hundred tokens the unpacking, which each tile of tokens repeats and whose warps
// wait half of the time, and what a shared tile's end costs (171 tokens, two tiles, 4096 features of 11008 columns: 20.7 us, 740 TFLOP/s).  Tokens loaded once for
// two neighbouring CTAs made it no faster (21.4 us, prompts 137).
//
// A sum takes all of a CTA's columns: the tensor core cuts its last bits off at each of K / 16 additions, a loss of 3.1e-6 of the result at
// 4096 columns and 9.8e-6 at 11008, which is what a product of bf16 matrices into fp32 loses in the library too.  Shorter sums
// need tensor memory that is not there, or outputs read and written several times.
//
// Every wait is bounded: a timeout sets MEDUSA_DEV_TIMEOUT, all roles stop, copies and products in
// flight are waited for and tensor memory is freed.
#include "linear_w4_tc.cuh"

namespace medusa {
namespace w4 {

namespace {

constexpr int kThreads = 768;              // W, products, x, products; 4 x 4 unpacking; 4 reading out
constexpr int kUnpackers = 16;
constexpr int kHalf = 128;                 // features of a half of a tile at most
constexpr int kMaxTN = 128;
constexpr int kMaxShare = 8;               // CTAs of a cluster
constexpr int kSlotsW = 4;
constexpr int kMaxSlotsX = 8;
constexpr uint32_t kHalfW = kHalf * kCols / 2;
constexpr uint32_t kOffScales = 2 * kHalfW;  // of a slot: the weights, scales [group][feature], zeros likewise
constexpr uint32_t kOffZeros = kOffScales + 2048;
constexpr uint32_t kSlotW = kOffZeros + 1024;

struct Tc {
  Args a;
  int TN, DN, NX;      // tokens of a tile, columns of a sum, slots of tokens (an even number)
  int halves, RH;      // halves of a tile and the features of one
  int mtiles, ntiles, kblocks;
  int share;           // CTAs of a cluster, which share a tile
  int grid;
  int slot_bytes;      // that come into a slot of weights
  int withhold;        // failure test: the first tokens are never loaded
};

// Tokens that each CTA of a cluster adds up.
__host__ __device__ constexpr int per_cta(int TN, int share) { return (TN / 4 + share - 1) / share * 4; }
static_assert((kMaxTN + 4 * kMaxShare) * 2 * kHalf * 4 <= kRing, "sums in the rings' place");

struct Tail {
  uint64_t w_full[kSlotsW], w_empty[kSlotsW], x_full[kMaxSlotsX], x_empty[kMaxSlotsX];
  uint64_t a_full[2][2], a_empty[2][2], d_full[2], d_empty[2], drain[2];
  uint32_t tmem;
  volatile int abort;
  int w_loads, x_loads;
};
constexpr uint32_t kSmem = kRing + sizeof(Tail);
static_assert(kSmem <= 232448, "shared memory of a CTA");

// A CTA's blocks, one after the other: feature tile, token tile, block of columns.
struct Walk {
  int mt, nt, kb, left;  // left: blocks, this one included
  int kb0, nb;           // the CTA's blocks of a tile
  int tile, stride;
  __device__ __forceinline__ void place(const Tc& p) {
    mt = tile / p.ntiles;
    nt = tile - mt * p.ntiles;
    kb = kb0;
  }
  __device__ __forceinline__ void next_tile(const Tc& p) {
    tile += stride;
    place(p);
  }
  __device__ __forceinline__ void step(const Tc& p) {
    --left;
    if (++kb == kb0 + nb) next_tile(p);
  }
};
__device__ __forceinline__ Walk walk_of(const Tc& p) {
  Walk x;
  const int tiles = p.mtiles * p.ntiles, rank = blockIdx.x % p.share;
  x.tile = blockIdx.x / p.share;
  x.stride = p.grid / p.share;
  x.kb0 = (int)((long long)p.kblocks * rank / p.share);
  x.nb = (int)((long long)p.kblocks * (rank + 1) / p.share) - x.kb0;
  x.left = (tiles - x.tile + x.stride - 1) / x.stride * x.nb;
  x.place(p);
  return x;
}

// Those of the blocks a thread unpacks, which are two apart.
template <int GROUPS>
struct Scales {
  Walk x;
  int row;
  size_t at, two;  // of the block; from it to the next but one of the same tile
  __device__ __forceinline__ void start(const Tc& p) { at = (size_t)(x.kb * GROUPS) * p.a.Nout + min(x.mt * (p.halves * p.RH) + row, p.a.Nout - 1); }
  __device__ __forceinline__ Scales(const Tc& p, const Walk& w, int r) : x(w), row(r), two((size_t)(2 * GROUPS) * p.a.Nout) { start(p); }
  __device__ __forceinline__ void next(const Tc& p) {
    if (x.kb + 2 < x.kb0 + x.nb) {
      x.left -= 2;
      x.kb += 2;
      at += two;
    } else {
      x.step(p);
      x.step(p);
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

template <int GROUPS, bool TILED>
__global__ void __launch_bounds__(kThreads, 1)
tc_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_s,
          const __grid_constant__ CUtensorMap tm_z, const __grid_constant__ Tc p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  Tail* tail = reinterpret_cast<Tail*>(smem + kRing);
  volatile int* abort = &tail->abort;
  if (smem_u32(smem) & 1023u) {  // the same in every thread
    if (threadIdx.x == 0) set_status(p.a.d_status, MEDUSA_DEV_TIMEOUT);
    return;
  }
  uint8_t* ring_x = smem + kSlotsW * kSlotW;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quads = (p.RH + 31) / 32;  // warps that have rows of a half
  if (threadIdx.x == 0) {
    tail->abort = 0;
    for (int i = 0; i < kSlotsW; ++i) {
      mbar_init(&tail->w_full[i], 1);
      mbar_init(&tail->w_empty[i], p.halves * quads);
    }
    for (int i = 0; i < p.NX; ++i) {
      mbar_init(&tail->x_full[i], 1);
      mbar_init(&tail->x_empty[i], p.halves);
    }
    for (int h = 0; h < 2; ++h) {
      for (int i = 0; i < 2; ++i) {
        mbar_init(&tail->a_full[h][i], quads);
        mbar_init(&tail->a_empty[h][i], 1);
      }
      mbar_init(&tail->d_full[h], 1);
      mbar_init(&tail->drain[h], 1);
      mbar_init(&tail->d_empty[h], quads);
    }
    fence_mbar_init();
  }
  if (warp == 1) {
    __syncwarp();
    tmem_alloc(&tail->tmem, kTmemCols);
    tmem_relinquish();
  }
  Walk x = walk_of(p);
  const int mt0 = x.mt, x0t = x.nt * p.TN;  // the one tile of a cluster
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
    for (Ring w; x.left > 0; x.step(p), w.next(kSlotsW), ++n) {
      if (w.used() && !warp_wait(&tail->w_empty[w.i], w.empty(), abort)) break;
      if (elect_one()) {
        mbar_expect_tx(&tail->w_full[w.i], (uint32_t)p.slot_bytes);
        tma_load_2d(smem + w.i * kSlotW, &tm_w, &tail->w_full[w.i], x.kb * (kCols / 2), x.mt * p.halves * p.RH);
        if (TILED) {
          tma_load_2d(smem + w.i * kSlotW + kOffScales, &tm_s, &tail->w_full[w.i], x.mt * p.halves * p.RH, x.kb * GROUPS);
          if (p.a.zeros) tma_load_2d(smem + w.i * kSlotW + kOffZeros, &tm_z, &tail->w_full[w.i], x.mt * p.halves * p.RH, x.kb * GROUPS);
        }
      }
      __syncwarp();
    }
    if (lane == 0) tail->w_loads = n;
  } else if (warp == 2) {
    // ------------------------------------------------------------ tokens
    int n = 0;
    for (Ring t; x.left > 0; x.step(p), t.next(p.NX), ++n) {
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
  } else if (warp == 1 || (warp == 3 && p.halves == 2)) {
    // ------------------------------------------------------------ products of half h
    // Issued by an elected lane of the whole warp, their addresses known to be the same in all lanes: by a lane on
    // its own a product took 80 clocks to issue, so 11.  What a block costs besides has to stay below what its products
    // take: one wait (an unpacking warp has waited for the tokens), and blocks two by two, whose buffers are constants.
    const int h = warp >> 1;
    const uint32_t idesc = uniform(idesc_bf16_f32(128, p.TN, false, false)), d = uniform(tmem + h * p.DN),
                   a0 = uniform(tmem + 2 * p.DN + h * 128), x0 = uniform((smem_u32(ring_x) >> 4) | (1u << 16)), half = uniform(p.TN * 8);
    const uint32_t full = smem_u32(&tail->a_full[h][0]);
    uint32_t slot = 0, phase = 0;  // of the tokens' ring; of the weights' buffers
    int k = 0, seg = 0;
    auto block = [&](auto buffer) {
      constexpr int B = decltype(buffer)::value;
      const uint32_t s = uniform(slot);
      if (k == 0 && seg > 0 && !warp_wait(&tail->d_empty[h], (uint32_t)(seg - 1) & 1u, abort)) return false;
      if (!warp_wait(full + 8 * B, phase, abort)) return false;
      tc_fence_after();
      if (elect_one()) {
        const uint32_t xd = x0 + s * 2 * half;
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          mma_bf16_ts(d, a0 + 64 * B + 8 * kk, desc_of(xd + (kk >> 2) * half + 2 * (kk & 3)), idesc, kk > 0 || k > 0);
        mma_commit(&tail->a_empty[h][B]);
        mma_commit(&tail->x_empty[s]);
        if (k == x.nb - 1) mma_commit(&tail->d_full[h]);
      }
      __syncwarp();
      slot = slot + 1 == (uint32_t)p.NX ? 0 : slot + 1;
      if (++k == x.nb) {
        k = 0;
        ++seg;
      }
      return true;
    };
    bool alive = true;
#pragma unroll 1
    for (int n = x.left; n > 0 && alive; n -= 2, phase ^= 1)
      alive = block(std::integral_constant<int, 0>()) && (n == 1 || block(std::integral_constant<int, 1>()));
    if (elect_one()) {
      // This warp's products and the arrivals they signal, before tensor and shared memory go away.
      mma_commit(&tail->drain[h]);
      mbar_wait_bounded(&tail->drain[h], 0, nullptr, kDrainNs);
    }
    __syncwarp();
  } else if (warp >= 4 && warp < 4 + kUnpackers && ((warp >> 2) & 1) < p.halves && (warp & 3) < quads) {
    // ------------------------------------------------------------ unpacking: half h, every second block, rows 32 q4 ..
    // A set has the blocks of one parity, and so the same slots of the ring and the same barriers each time: it
    // passes over no phase of them.
    const int h = (warp >> 2) & 1, set = warp >= 4 + kUnpackers / 2, q4 = warp & 3, row = 32 * q4 + lane;
    const uint32_t to = tmem + ((uint32_t)(32 * q4) << 16) + 2 * p.DN + h * 128 + set * 64;
    const uint32_t sw = 16 * ((row >> 1) & 3);  // 64-byte swizzle
    const uint32_t free = smem_u32(&tail->a_empty[h][set]), filled = smem_u32(&tail->a_full[h][set]), tokens = smem_u32(&tail->x_full[0]);
    uint32_t free_phase = 1, slot = set, x_slot = set, x_round = 0;
    bool first = true;  // the buffer was never used
    uint32_t round = 0;
    const int rows = p.halves * p.RH;
    if (set) x.step(p);
    int left = x.left;
    Scales<GROUPS> scales(p, x, h * p.RH + row);
    Raw<GROUPS> raw{};
    if (!TILED) raw = scales.load(p);
#pragma unroll 1
    for (; left > 0; left -= 2) {
      Group g[GROUPS];
      if (!TILED) {
#pragma unroll
        for (int k = 0; k < GROUPS; ++k) g[k] = group_of(raw.s[k], raw.z[k]);
        scales.next(p);
        raw = scales.load(p);  // of the set's next block: they take a round trip to memory
      }
      if (!warp_wait(smem_u32(&tail->w_full[0]) + 8 * slot, round, abort)) break;
      if (TILED) {
        const uint8_t* at = smem + slot * kSlotW + kOffScales;
#pragma unroll
        for (int k = 0; k < GROUPS; ++k) {
          const int i = k * rows + h * p.RH + row;
          g[k] = group_of(reinterpret_cast<const uint16_t*>(at)[i], p.a.zeros ? at[kOffZeros - kOffScales + i] : 8);
        }
      }
      const uint32_t w = smem_u32(smem) + slot * kSlotW + (h * p.RH + row) * 64;
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
      if (q4 == 0) {  // for the warp that issues the products
        if (!warp_wait(tokens + 8 * x_slot, x_round, abort)) break;
        x_slot += 2;
        if (x_slot >= (uint32_t)p.NX) {
          x_slot -= p.NX;
          x_round ^= 1;
        }
      }
      warp_arrive(filled, lane);
    }
  } else if (warp >= 4 + kUnpackers && p.share == 1 && (warp & 3) < quads) {
    // ------------------------------------------------------------ reading out
    const int q4 = warp & 3, m = 32 * q4 + lane;
    const uint32_t lanes = tmem + ((uint32_t)(32 * q4) << 16);
    bool alive = true;
    for (int seg = 0; x.left > 0 && alive; ++seg, x.left -= x.nb, x.next_tile(p)) {
      const int t0 = x.nt * p.TN, tokens = min(p.TN, p.a.T - t0);
      for (int h = 0; h < p.halves; ++h) {
        if (!(alive = warp_wait(&tail->d_full[h], seg & 1, abort))) break;
        tc_fence_after();
        const int n = (x.mt * p.halves + h) * p.RH + m;
        const bool mine = m < p.RH && n < p.a.Nout;
        size_t at = (size_t)t0 * p.a.Nout + n;
#pragma unroll 1
        for (int c = 0; c < tokens; c += 16) {
          float v[16];
          __syncwarp();
          tmem_ld16(lanes + h * p.DN + c, v);
          tmem_wait_ld();
          if (!mine) continue;
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
        __syncwarp();
        tc_fence_before();
        warp_arrive(smem_u32(&tail->d_empty[h]), lane);
      }
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
  if (p.share > 1) {
    // The tile's sums, of which each CTA of the cluster has a part: CTA r's tokens' sums go to CTA r, into the rings'
    // place, [sender][four tokens][feature][4].
    const int rank = blockIdx.x % p.share, per = per_cta(p.TN, p.share), rows = p.halves * p.RH;
    const int h = (warp >> 2) & 1, part = warp >= 4 + kUnpackers / 2, m = 32 * (warp & 3) + lane;
    const bool works = warp >= 4 && warp < 4 + kUnpackers && h < p.halves && (warp & 3) < quads;
    const uint32_t mine = 16 * (h * p.RH + m);
    cluster_sync();  // all products of the cluster are done, and nobody reads from the rings
    if (works) {
      const uint32_t from = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + h * p.DN, at = smem_u32(smem) + mine;
#pragma unroll 1
      for (int c = 16 * part; c < p.TN; c += 32) {
        float v[16];
        __syncwarp();
        tmem_ld16(from + c, v);
        tmem_wait_ld();
        if (m >= p.RH) continue;
        int to = c / per, col = c - to * per;
#pragma unroll
        for (int e = 0; e < 16; e += 4) {
          uint32_t there;
          asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(at + 4 * ((rank * per + col) * rows)), "r"(to));
          asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(there), "f"(v[e]), "f"(v[e + 1]), "f"(v[e + 2]), "f"(v[e + 3])
                       : "memory");
          col += 4;
          if (col == per) {
            col = 0;
            ++to;
          }
        }
      }
    }
    cluster_sync();
    const int tokens = min(per, min(p.TN - rank * per, p.a.T - x0t - rank * per)), n = mt0 * rows + h * p.RH + m;
    if (works && m < p.RH && n < p.a.Nout)
      for (int t = 4 * part; t < tokens; t += 8) {
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int r = 0; r < p.share; ++r) {
          const float4 w = *reinterpret_cast<const float4*>(smem + 4 * ((r * per + t) * rows) + mine);
          v.x += w.x;
          v.y += w.y;
          v.z += w.z;
          v.w += w.w;
        }
        const float y[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (t + e < tokens) store_y(p.a, x0t + rank * per + t + e, n, y[e]);
      }
  }
  if (warp == 1) {
    __syncwarp();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// ------------------------------------------------------------------ host side

static int log2_of(int n) { return n > 1 ? 1 + log2_of(n / 2) : 0; }

static Tc plan(int T, int K, int Nout) {
  Tc best{};
  double least = 0;
  const int kblocks = (K + kCols - 1) / kCols;
  for (int share = 1; share <= kMaxShare && share <= kblocks; share *= 2) {
    Tc p{};
    p.ntiles = ceil_div(T, kMaxTN);  // in 64 bits: T may be nearly 2^31
    p.TN = (ceil_div(T, p.ntiles) + 15) / 16 * 16;
    p.ntiles = ceil_div(T, p.TN);
    p.DN = (p.TN + 31) / 32 * 32;
    p.NX = (int)((kRing - kSlotsW * kSlotW) / (p.TN * 256)) & ~1;
    if (p.NX > kMaxSlotsX) p.NX = kMaxSlotsX;
    p.kblocks = kblocks;
    p.share = share;
    // Rounds that the tiles need when they are as high as can be, then the tiles that fill these rounds.
    const int at_once = clusters_at_once(share);
    const long long fewest = (long long)((Nout + 2 * kHalf - 1) / (2 * kHalf)) * p.ntiles, rounds = (fewest + at_once - 1) / at_once;
    if (share > 1 && rounds > 1) break;
    const long long high = rounds * at_once / p.ntiles;
    int rows = (int)((Nout + high - 1) / high);
    p.halves = rows > kHalf ? 2 : 1;
    p.RH = ((rows + p.halves - 1) / p.halves + 15) / 16 * 16;
    p.mtiles = (Nout + p.halves * p.RH - 1) / (p.halves * p.RH);
    const long long tiles = (long long)p.mtiles * p.ntiles;
    p.grid = (int)(tiles < at_once ? tiles : at_once) * share;
    // Clocks: a block's products, what its way through the two sets of unpacking warps takes, and its bytes, whichever is
    // most (as measured these come to 36 a clock: 112 features x 96 tokens 864 clocks, 160 x 128 1240, 256 x 128
    // 1380); what a tile's end costs, and the exchange of sums (171 tokens x 4096 features of 11008 columns: tiles of 256
    // features that four CTAs share 20.7 us, of 112 that two share 23.0).
    const double products = 4.0 * p.TN * p.halves, bytes = (p.halves * p.RH * 64 + p.TN * 256) / 36.0;
    double block = products > 850 ? products : 850;
    if (bytes > block) block = bytes;
    const double cost = (double)rounds * ((kblocks + share - 1) / share * block + 1500 + (share > 1 ? 2000 * log2_of(share) + p.TN * p.halves * p.RH / 1.6 : 0));
    if (least == 0 || cost < least) {
      least = cost;
      best = p;
    }
  }
  return best;
}

}  // namespace

Division tc_division(int T, int K, int Nout) {
  const Tc p = plan(T, K, Nout);
  return {p.share, p.TN, p.halves * p.RH, p.mtiles * p.ntiles, p.grid};
}

medusa_status tc_launch(const Args& a, int withhold, cudaStream_t s) {
  if (!encode_fn()) return MEDUSA_ERR_CUDA;
  Tc p = plan(a.T, a.K, a.Nout);
  p.a = a;
  p.withhold = withhold;
  const int per = kCols >> a.glog, ng = a.K >> a.glog, rows = p.halves * p.RH;
  const bool tiled = a.Nout % 16 == 0 && aligned16(a.scales) && aligned16(a.zeros);
  p.slot_bytes = rows * (kCols / 2 + (tiled ? per * (a.zeros ? 3 : 2) : 0));
  CUtensorMap mw, mx, ms, mz;
  if (!make_map(&mw, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.q, a.K / 2, a.Nout, a.K / 2, kCols / 2, rows, CU_TENSOR_MAP_SWIZZLE_64B) ||
      !make_map(&mx, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.x, a.K, a.T, a.ldx * 2, 64, p.TN, CU_TENSOR_MAP_SWIZZLE_128B))
    return MEDUSA_ERR_CUDA;
  ms = mz = mw;
  if (tiled && (!make_map(&ms, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.scales, a.Nout, ng, (long long)a.Nout * 2, rows, per, CU_TENSOR_MAP_SWIZZLE_NONE) ||
                (a.zeros && !make_map(&mz, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.zeros, a.Nout, ng, a.Nout, rows, per, CU_TENSOR_MAP_SWIZZLE_NONE))))
    return MEDUSA_ERR_CUDA;
  auto kern = a.glog == 5 ? (tiled ? tc_kernel<4, true> : tc_kernel<4, false>)
              : a.glog == 6 ? (tiled ? tc_kernel<2, true> : tc_kernel<2, false>)
                            : (tiled ? tc_kernel<1, true> : tc_kernel<1, false>);
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem) != cudaSuccess) return MEDUSA_ERR_CUDA;
  launch_clusters(kern, p.grid, kThreads, kSmem, p.share, s, mw, mx, ms, mz, p);
  return launch_status();
}

}  // namespace w4
}  // namespace medusa
