// medusa_linear_w4 on tcgen05 tensor cores: up to 64 tokens, and more of a small layer in tiles of up to 64, bound by memory and
// by the unpacking of the weights.
//
// As in the kernel for many tokens (linear_w4_tc.cu) weights come as they are kept by TMA and sixteen warps unpack
// them into tensor memory, the products' first operand.  A block of 128 columns of 128 features costs an SM's
// schedulers some 350 clocks of unpacking each, so that what counts is that all of them have the same number of
// blocks: the tiles of 128 features and up to 64 tokens that a cluster of CTAs has, laid end to end, are divided evenly over its CTAs (64
// tokens, 22016 features of 4096 columns: 17.8 us, 2.8 TB/s; tiles of up to 256 features in whole rounds 22.4).  A CTA has its whole tiles first and
// then the parts of tiles, whose sums stay in tensor memory until the end and then go through distributed shared
// memory to the tile's CTAs, which add up some tokens each, in the CTAs' order.
//
// Loads bring two blocks (256 columns) at a time.  A load costs the warp that starts it some 130 clocks whatever its size,
// which with weights, scales, zeros and twice 64 columns of tokens for each block was more than the block's unpacking (17
// tokens, 128256 features: 72 us; now 59, 4.6 TB/s).  Of the 500 clocks or so that a block takes now the
// schedulers issue in half: the rest is sixteen warps waiting for loads, tensor memory and one another.
//
// Within a CTA four sets of four warps unpack a block each into a buffer of their own, and two warps issue the
// products of every second block, each into sums of its own: what lies between a block's products and the next
// one's (some 800 clocks) passes under the other's.  The sums are added as they are read out.  The tensor core cuts
// a sum's last bits off, so that what is lost grows with the products that are added to it: of up to 16 tokens a
// stream's blocks go to four sums in turn, of up to 32 to two (4096 columns, one token: an error of 2.9e-7 of the
// result, with one sum each 1.4e-6).
//
// Every wait is bounded, as there.
#include <atomic>

#include "linear_w4_tc.cuh"

namespace medusa {
namespace w4 {
namespace {

constexpr int kThreads = 768;           // W, products, x, products; 4 x 4 unpacking; 4 reading out
constexpr int kRows = 128;              // features of a tile at most
constexpr int kMaxTN = 64;
constexpr int kMaxShare = 8;            // CTAs of a cluster
constexpr int kSets = 4, kSlots = 4;    // of both rings, of two blocks each
constexpr uint32_t kSums = 64;           // columns of tensor memory that a part's sums of one stream have
constexpr uint32_t kOffScales = kRows * kCols;  // of a slot: the weights, scales [group][feature], zeros likewise
constexpr uint32_t kOffZeros = kOffScales + 2048;
constexpr uint32_t kSlotW = kOffZeros + 1024;
constexpr uint32_t kRegion = (kMaxTN + 4 * kMaxShare) * kRows * 4;  // sums that the CTAs of a cluster send to one another
static_assert(kSlotW % 1024 == 0, "the swizzled tiles' alignment");
static_assert(kSlots * (kSlotW + kMaxTN * 512) <= kRing && 2 * kRegion <= kRing, "shared memory of a CTA");

struct Plan {
  Args a;
  int TN, DN, RH;       // tokens of a tile, columns of a sum, features of a tile
  int turns;            // sums of a stream, which take its blocks in turn
  int tiles, ntiles;    // all tiles; those of the same features, one after the other
  int kpairs;           // pairs of blocks of K
  int slabs;            // 64 columns of tokens that a load brings: 4, or 1 if K has other columns than multiples of 64
  int share, each;      // CTAs of a cluster, tiles of one
  int clusters;
  int slot_bytes;       // that come into a slot of weights
  long long cost;       // clocks
  int withhold;         // failure test: the first tokens are never loaded
};

// A part of a tile: [0] is the part that a CTA's range begins with, [1] the one that it ends with.
struct Part {
  int there, n0, t0;            // whether there is one; its features and tokens
  int order, turns;             // where the CTA's walk has it; sums of a stream
  int n, sender, per;           // CTAs that share the tile, which of them this is, tokens of each
  int region;                   // where their sums arrive
  uint2 to[kMaxTN / 4];         // of four tokens: the CTA of the cluster that adds them up, where in its shared memory
};

struct Tail {
  Part part[2];
  uint64_t w_full[kSlots], w_empty[kSlots], x_full[kSlots], x_empty[kSlots];
  uint64_t a_full[kSets], a_empty[kSets], drain[2];
  // Of even and odd parts, by stream.  One barrier for both could be two phases ahead of who waits for it, which looks
  // like none.
  uint64_t d_full[2][2], d_empty[2][2];
  uint32_t tmem;
  volatile int abort;
  int w_loads, x_loads;
};
constexpr uint32_t kSmem = kRing + sizeof(Tail);
static_assert(kSmem <= 232448, "shared memory of a CTA");

// The cluster's pairs of blocks: those of its first tile, its second, ...; CTA j of it has [begin(j), begin(j + 1)).
struct Range {
  int tile0;
  uint32_t total, share, log2;
  __device__ __forceinline__ uint32_t begin(uint32_t j) const { return total * j >> log2; }
  __device__ __forceinline__ uint32_t owner(uint32_t pair) const { return ((pair + 1) * share - 1) / total; }
};
// A CTA's pairs of blocks, one after the other: whole tiles, the part of a tile that its range ends with, and last the part that it
// begins with.  So the sums of both parts may stay where they are until the end.
struct Walk {
  int mt, nt, kp, left;          // tile of features, of tokens, pair; left: pairs, this one included
  int mt0, nt0, kp0, first;      // the part that comes last: where it is, its pairs (0: none)
  __device__ __forceinline__ void to_first() {
    if (left == first) {
      mt = mt0;
      nt = nt0;
      kp = kp0;
    }
  }
  __device__ __forceinline__ void next_tile(int ntiles) {
    kp = 0;
    if (++nt == ntiles) {
      nt = 0;
      ++mt;
    }
  }
  __device__ __forceinline__ void step(const Plan& p) {
    --left;
    if (++kp == p.kpairs) next_tile(p.ntiles);
    to_first();
  }
  // Pairs of the tile that the walk is in, all of them if they are whole tiles'.
  __device__ __forceinline__ int part(int kpairs) const { return left <= first ? left : min(left - first, kpairs); }
  __device__ __forceinline__ void next_part(const Plan& p, int np) {
    left -= np;
    next_tile(p.ntiles);
    to_first();
  }
};

template <int GROUPS>
__device__ __forceinline__ Raw<GROUPS> load_groups(const Plan& p, const Walk& x, int odd, int row) {
  Raw<GROUPS> r;
  const int kb = 2 * x.kp + odd;
  const size_t at = (size_t)kb * GROUPS * p.a.Nout + min(x.mt * p.RH + row, p.a.Nout - 1);
#pragma unroll
  for (int i = 0; i < GROUPS; ++i) {
    r.s[i] = 0;  // behind the last column: weights of 0
    r.z[i] = 8;
    if (x.left > 0 && kb * kCols + kCols / GROUPS * i < p.a.K) {
      r.s[i] = p.a.scales[at + (size_t)i * p.a.Nout];
      if (p.a.zeros) r.z[i] = p.a.zeros[at + (size_t)i * p.a.Nout];
    }
  }
  return r;
}

// 16 columns of a part's sum, that of all its sums: of both streams, `used` of each.
__device__ __forceinline__ void read_sums(uint32_t at, int DN, int used, float* v) {
  float w[16];
  __syncwarp();
  tmem_ld16(at, v);
  tmem_ld16(at + kSums, w);
  tmem_wait_ld();
#pragma unroll
  for (int e = 0; e < 16; ++e) v[e] += w[e];
#pragma unroll 1
  for (int i = 1; i < used; ++i) {
    float u[16];
    __syncwarp();
    tmem_ld16(at + i * DN, u);
    tmem_ld16(at + kSums + i * DN, w);
    tmem_wait_ld();
#pragma unroll
    for (int e = 0; e < 16; ++e) v[e] += u[e] + w[e];
  }
}

template <int GROUPS, bool TILED>
__global__ void __launch_bounds__(kThreads, 1)
stream_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_s,
              const __grid_constant__ CUtensorMap tm_z, const __grid_constant__ Plan p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  Tail* tail = reinterpret_cast<Tail*>(smem + kRing);
  volatile int* abort = &tail->abort;
  if (smem_u32(smem) & 1023u) {  // the same in every thread of every CTA
    if (threadIdx.x == 0) set_status(p.a.d_status, MEDUSA_DEV_TIMEOUT);
    return;
  }
  uint8_t* ring_x = smem + kSlots * kSlotW;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quads = (p.RH + 31) / 32;  // warps that have rows of a tile
  if (threadIdx.x == 0) {
    tail->abort = 0;
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&tail->w_full[i], 1);
      mbar_init(&tail->w_empty[i], 2 * quads);
    }
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&tail->x_full[i], 1);
      mbar_init(&tail->x_empty[i], 2);
    }
    for (int i = 0; i < kSets; ++i) {
      mbar_init(&tail->a_full[i], quads);
      mbar_init(&tail->a_empty[i], 1);
    }
    for (int s = 0; s < 2; ++s) {
      for (int k = 0; k < 2; ++k) {
        mbar_init(&tail->d_full[k][s], 1);
        mbar_init(&tail->d_empty[k][s], quads);
      }
      mbar_init(&tail->drain[s], 1);
    }
    fence_mbar_init();
  }
  if (warp == 1) {
    __syncwarp();
    tmem_alloc(&tail->tmem, kTmemCols);
    tmem_relinquish();
  }
  const int rank = blockIdx.x % p.share, tile0 = blockIdx.x / p.share * p.each;
  const Range range{tile0, (uint32_t)(min(p.each, p.tiles - tile0) * p.kpairs), (uint32_t)p.share, (uint32_t)__ffs(p.share) - 1};
  const int begin = (int)range.begin(rank), end = (int)range.begin(rank + 1);
  const int lead = begin % p.kpairs;  // pairs of the first tile that are another CTA's
  const int first = lead ? min(p.kpairs - lead, end - begin) : 0;
  const int whole = tile0 + (begin + first) / p.kpairs, last = tile0 + begin / p.kpairs;  // tiles that the walk begins and ends with
  Walk x{whole / p.ntiles, whole % p.ntiles, 0, end - begin, last / p.ntiles, last % p.ntiles, lead, first};
  x.to_first();
  const int parts = (first > 0) + (end - begin - first + p.kpairs - 1) / p.kpairs, tail_pairs = (end - begin - first) % p.kpairs;
  if (warp == 2 && p.share > 1) {
    // The divisions of the end, here where the kernel in front may still be running.
    const int k = lane >> 4, tile = (k ? end - 1 : begin) / p.kpairs, f = (int)range.owner(tile * p.kpairs);
    const int n = (int)range.owner((tile + 1) * p.kpairs - 1) - f + 1, per = (p.TN / 4 + n - 1) / n * 4;
    const auto region = [&](int r) { return (int)range.begin(r) / p.kpairs == tile ? 0u : kRegion; };
    Part& part = tail->part[k];
    if ((lane & 15) == 0) {
      part.there = k ? tail_pairs > 0 : first > 0;
      part.n0 = (tile0 + tile) / p.ntiles * p.RH;
      part.t0 = (tile0 + tile) % p.ntiles * p.TN;
      part.order = parts - 1 - (k && first ? 1 : 0);
      part.turns = min(k ? tail_pairs : first, p.turns);
      part.n = n;
      part.sender = rank - f;
      part.per = per;
      part.region = (int)region(rank);
    }
    const int t = 4 * (lane & 15), j = min(t / per, n - 1);  // tokens from p.TN on belong to nobody
    part.to[lane & 15] = make_uint2(f + j, region(f + j) + 4 * ((rank - f) * per + t - j * per) * p.RH);
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch(&tm_w);
    tma_prefetch(&tm_x);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_wait();
  pdl_trigger();
  const uint32_t tmem = tail->tmem, weights = tmem + 4 * kSums;  // sums: [part, even or odd][stream][turn]; then unpacked weights

  if (warp == 0) {
    // ------------------------------------------------------------ weights as they are kept
    int n = 0;
    for (Ring w; x.left > 0; x.step(p), w.next(kSlots), ++n) {
      if (w.used() && !warp_wait(&tail->w_empty[w.i], w.empty(), abort)) break;
      if (elect_one()) {
        uint8_t* to = smem + w.i * kSlotW;
        const int row = x.mt * p.RH;
        mbar_expect_tx(&tail->w_full[w.i], (uint32_t)p.slot_bytes);
        tma_load_2d(to, &tm_w, &tail->w_full[w.i], x.kp * kCols, row);
        if (TILED) {
          tma_load_2d(to + kOffScales, &tm_s, &tail->w_full[w.i], row, x.kp * (2 * GROUPS));
          if (p.a.zeros) tma_load_2d(to + kOffZeros, &tm_z, &tail->w_full[w.i], row, x.kp * (2 * GROUPS));
        }
      }
      __syncwarp();
    }
    if (lane == 0) tail->w_loads = n;
  } else if (warp == 2) {
    // ------------------------------------------------------------ tokens
    int n = 0;
    for (Ring t; x.left > 0; x.step(p), t.next(kSlots), ++n) {
      if (t.used() && !warp_wait(&tail->x_empty[t.i], t.empty(), abort)) break;
      if (elect_one()) {
        mbar_expect_tx(&tail->x_full[t.i], (uint32_t)p.TN * 512);
        uint8_t* const to = ring_x + t.i * (p.TN * 512);
        const int t0 = x.nt * p.TN;
        if (p.slabs == 4) {
          if (!(p.withhold && n == 0)) tma_load_3d(to, &tm_x, &tail->x_full[t.i], 0, t0, x.kp * 4);
        } else {
          for (int u = 0; u < 4; ++u)
            if (!(p.withhold && n == 0 && u == 0))
              tma_load_2d(to + u * (p.TN * 128), &tm_x, &tail->x_full[t.i], x.kp * (2 * kCols) + u * 64, t0);
        }
      }
      __syncwarp();
    }
    if (lane == 0) tail->x_loads = n;
  } else if (warp == 1 || warp == 3) {
    // ------------------------------------------------------------ products of stream s
    const int s = warp >> 1;
    const uint32_t idesc = uniform(idesc_bf16_f32(128, p.TN, false, false)), a0 = uniform(weights),
                   x0 = uniform((smem_u32(ring_x) >> 4) | (1u << 16)), half = uniform(p.TN * 8);
    const uint32_t full = smem_u32(&tail->a_full[0]);
    uint32_t i = 0;  // pairs
    bool alive = true;
    for (int part = 0; x.left > 0 && alive; ++part) {
      const int np = x.part(p.kpairs);
      const uint32_t d = uniform(tmem + (2 * (part & 1) + s) * kSums);
      if (part > 1 && !(alive = warp_wait(&tail->d_empty[part & 1][s], (uint32_t)(part / 2 - 1) & 1u, abort))) break;  // the part before the last is read out
      const uint32_t last = i + np;
#pragma unroll 1
      for (uint32_t own = 0; i < last; ++i, ++own) {
        const uint32_t set = uniform(2 * (i & 1) + s), slot = uniform(i % kSlots), sum = uniform(d + (own & (p.turns - 1)) * p.DN);
        if (!(alive = warp_wait(full + 8 * set, (i / 2) & 1u, abort))) break;
        tc_fence_after();
        if (elect_one()) {
          const uint32_t xd = x0 + (4 * slot + 2 * s) * half, a = a0 + 64 * set;
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            mma_bf16_ts(sum, a + 8 * kk, desc_of(xd + (kk >> 2) * half + 2 * (kk & 3)), idesc, kk > 0 || own >= (uint32_t)p.turns);
          mma_commit(&tail->a_empty[set]);
          mma_commit(&tail->x_empty[slot]);
        }
        __syncwarp();
      }
      if (!alive) break;
      if (elect_one()) mma_commit(&tail->d_full[part & 1][s]);
      __syncwarp();
      x.next_part(p, np);
    }
    if (elect_one()) {
      // This warp's products and the arrivals they signal, before tensor and shared memory go away.
      mma_commit(&tail->drain[s]);
      mbar_wait_bounded(&tail->drain[s], 0, nullptr, kDrainNs);
    }
    __syncwarp();
  } else if (warp >= 4 && warp < 4 + 4 * kSets && (warp & 3) < quads) {
    // ------------------------------------------------------------ unpacking: a block of every second pair, rows 32 q4 ..
    const int set = (warp - 4) >> 2, odd = set & 1, q4 = warp & 3, row = 32 * q4 + lane;
    const uint32_t to = weights + ((uint32_t)(32 * q4) << 16) + 64 * set;
    const uint32_t sw = 16 * (row & 7);  // 128-byte swizzle
    const uint32_t free = smem_u32(&tail->a_empty[set]), filled = smem_u32(&tail->a_full[set]), tokens = smem_u32(&tail->x_full[0]),
                   came = smem_u32(&tail->w_full[0]), left_empty = smem_u32(&tail->w_empty[0]);
    uint32_t phase = 0;  // of the set's blocks
    const int pairs = x.left;
    if (set > 1) x.step(p);
    Raw<GROUPS> raw{};
    if (!TILED) raw = load_groups<GROUPS>(p, x, odd, row);
#pragma unroll 1
    for (int i = set >> 1; i < pairs; i += 2) {
      Group g[GROUPS];
      if (!TILED) {
#pragma unroll
        for (int k = 0; k < GROUPS; ++k) g[k] = group_of(raw.s[k], raw.z[k]);
        x.step(p);
        x.step(p);
        raw = load_groups<GROUPS>(p, x, odd, row);  // of the set's next block: they take a round trip to memory
      }
      const uint32_t slot = (uint32_t)i % kSlots, round = (uint32_t)i / kSlots & 1u;
      if (!warp_wait(came + 8 * slot, round, abort)) break;
      if (q4 == 0 && !warp_wait(tokens + 8 * slot, round, abort)) break;  // for the warp that issues the products
      const uint8_t* at = smem + slot * kSlotW;
      if (TILED) {
#pragma unroll
        for (int k = 0; k < GROUPS; ++k) {
          const int e = (odd * GROUPS + k) * p.RH + row;
          g[k] = group_of(reinterpret_cast<const uint16_t*>(at + kOffScales)[e], p.a.zeros ? at[kOffZeros + e] : 8);
        }
      }
      const uint32_t w = smem_u32(at) + row * 128;
      uint4 v[4];
#pragma unroll
      for (int c = 0; c < 4; ++c)
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v[c].x), "=r"(v[c].y), "=r"(v[c].z), "=r"(v[c].w) : "r"(w + ((64 * odd + 16 * c) ^ sw)) : "memory");
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
      warp_arrive(left_empty + 8 * slot, lane);
      if (i > 1 && !warp_wait(free, phase ^ 1, abort)) break;
      tc_fence_after();
      tmem_st32u(to, r);
      half_block(1);
      __syncwarp();
      tmem_st32u(to + 32, r);
      tmem_wait_st();
      tc_fence_before();
      warp_arrive(filled, lane);
      phase ^= 1;
    }
  } else if (warp >= 4 + 4 * kSets && (warp & 3) < quads) {
    // ------------------------------------------------------------ whole tiles, read out
    const int q4 = warp & 3, m = 32 * q4 + lane;
    for (int part = 0; x.left > 0; ++part) {
      const int np = x.part(p.kpairs), n = x.mt * p.RH + m, t0 = x.nt * p.TN, tokens = min(p.TN, p.a.T - t0);
      if (np < p.kpairs) break;  // what is left are parts
      uint64_t* const full = tail->d_full[part & 1];
      if (!(warp_wait(full, (uint32_t)(part / 2) & 1u, abort) && warp_wait(full + 1, (uint32_t)(part / 2) & 1u, abort))) break;
      tc_fence_after();
      const uint32_t at = tmem + ((uint32_t)(32 * q4) << 16) + 2 * (part & 1) * kSums;
      const bool mine = m < p.RH && n < p.a.Nout;
      size_t to = (size_t)t0 * p.a.Nout + n;
#pragma unroll 1
      for (int c = 0; c < tokens; c += 16) {
        float v[16];
        read_sums(at + c, p.DN, min(np, p.turns), v);
        if (!mine) continue;
        const int more = tokens - c;
        if (p.a.y32) {
          float* y = static_cast<float*>(p.a.y);
#pragma unroll
          for (int e = 0; e < 16; ++e, to += p.a.Nout)
            if (e < more) y[to] = v[e];
        } else {
          uint16_t* y = static_cast<uint16_t*>(p.a.y);
#pragma unroll
          for (int e = 0; e < 16; ++e, to += p.a.Nout)
            if (e < more) y[to] = bf16_rn(v[e]);
        }
      }
      __syncwarp();
      tc_fence_before();
      for (int s = 0; s < 2; ++s) warp_arrive(smem_u32(&tail->d_empty[part & 1][s]), lane);
      x.next_part(p, np);
    }
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (threadIdx.x == 0 && *abort) {
    set_status(p.a.d_status, MEDUSA_DEV_TIMEOUT);
    // No copy may land after exit: wait (bounded) for the last phase of every load.
    for (int i = max(0, tail->w_loads - kSlots); i < tail->w_loads; ++i)
      mbar_wait_bounded(&tail->w_full[i % kSlots], (uint32_t)(i / kSlots) & 1u, nullptr, kDrainNs);
    for (int i = max(0, tail->x_loads - kSlots); i < tail->x_loads; ++i)
      mbar_wait_bounded(&tail->x_full[i % kSlots], (uint32_t)(i / kSlots) & 1u, nullptr, kDrainNs);
  }
  if (p.share > 1) {
    // Parts of tiles.  The sums go into the rings' place, [sender][four tokens][feature][4]: a store of 16 bytes a lane
    // takes no longer than one of 4.
    const int m = 32 * (warp & 3) + lane, group = (warp - 4) >> 2;  // a feature, and which of the tokens
    const bool works = warp >= 4 && warp < 4 + 4 * kSets && m < p.RH;
    cluster_sync();  // all products of the cluster are done, and nobody reads from the rings
    if (warp >= 4 && warp < 4 + 4 * kSets && (warp & 3) < quads) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const Part& part = tail->part[k];
        if (!part.there) continue;
        const uint32_t from = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + 2 * (part.order & 1) * kSums;
#pragma unroll 1
        for (int c = 16 * group; c < p.TN; c += 16 * kSets) {
          float v[16];
          read_sums(from + c, p.DN, part.turns, v);
          if (!works) continue;
#pragma unroll
          for (int e = 0; e < 16; e += 4) {
            const uint2 to = part.to[(c + e) / 4];
            uint32_t there;
            asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(smem_u32(smem) + to.y + 16 * m), "r"(to.x));
            asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(there), "f"(v[e]), "f"(v[e + 1]), "f"(v[e + 2]), "f"(v[e + 3])
                         : "memory");
          }
        }
      }
    }
    cluster_sync();
    if (works)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const Part& part = tail->part[k];
        if (!part.there) continue;
        const int skip = part.sender * part.per, t0 = part.t0 + skip;
        const int tokens = min(min(part.per, p.TN - skip), p.a.T - t0), n = part.n0 + m;
        const float4* sums = reinterpret_cast<const float4*>(smem + part.region) + m;
        for (int t = 4 * group; t < tokens; t += 4 * kSets) {
          float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
          for (int r = 0; r < part.n; ++r) {
            const float4 w = sums[(r * part.per + t) / 4 * p.RH];
            v.x += w.x;
            v.y += w.y;
            v.z += w.z;
            v.w += w.w;
          }
          const float y[4] = {v.x, v.y, v.z, v.w};
          if (n < p.a.Nout)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (t + e < tokens) store_y(p.a, t0 + t + e, n, y[e]);
        }
      }
  }
  if (warp == 1) {
    __syncwarp();
    tmem_dealloc(tmem, kTmemCols);
  }
}

static Plan plan(int T, int K, int Nout) {
  Plan best{};
  for (int share = 1; share <= kMaxShare; share *= 2) {
    Plan p{};
    p.ntiles = ceil_div(T, kMaxTN);  // in 64 bits: T may be nearly 2^31
    p.TN = (ceil_div(T, p.ntiles) + 15) / 16 * 16;
    p.ntiles = ceil_div(T, p.TN);
    p.DN = p.TN > 32 ? 64 : p.TN;
    p.turns = kSums / p.DN;
    p.RH = Nout >= kRows ? kRows : (Nout + 15) / 16 * 16;
    p.kpairs = (K + 2 * kCols - 1) / (2 * kCols);
    p.slabs = K % 64 ? 1 : 4;
    p.share = share;
    const long long tiles = (long long)((Nout + p.RH - 1) / p.RH) * p.ntiles;
    if (share > p.kpairs || tiles * p.kpairs * kMaxShare > 0x7fffffffll) break;
    p.tiles = (int)tiles;
    const int n = clusters_at_once(share);
    p.each = (p.tiles + n - 1) / n;
    p.clusters = (p.tiles + p.each - 1) / p.each;
    // Clocks: of a pair of blocks, and of the exchange of sums.
    p.cost = ((long long)p.each * p.kpairs + share - 1) / share * 900 + (share > 1 ? 3000 : 0);
    if (best.tiles == 0 || p.cost < best.cost) best = p;
  }
  return best;
}

// Tokens as [64 columns][token][...], so that one load brings four times 64 columns of all.
static bool make_slabs(CUtensorMap* m, const Args& a, int TN) {
  const cuuint64_t dims[3] = {64, (cuuint64_t)a.T, (cuuint64_t)(a.K / 64)}, strides[2] = {(cuuint64_t)a.ldx * 2, 128};
  const cuuint32_t box[3] = {64, (cuuint32_t)TN, 4}, one[3] = {1, 1, 1};
  return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(static_cast<const void*>(a.x)), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                     CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

int clusters_at_once(int share) {
  static std::atomic<int> known[16][4];
  if (share == 1) return device_sm_count();
  int dev = 0;
  const int k = share == 2 ? 1 : share == 4 ? 2 : 3;
  const int otherwise = device_sm_count() * 3 / 4 / share;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 16) return otherwise;
  int n = known[dev][k].load(std::memory_order_relaxed);
  if (n) return n;
  auto kern = stream_kernel<1, true>;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(share);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = share;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem) != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n < 1) {
    cudaGetLastError();
    n = otherwise;
  }
  known[dev][k].store(n, std::memory_order_relaxed);
  return n;
}

int stream_blocks(int T, int K, int Nout) {
  const Plan p = plan(T, K, Nout);
  return p.share ? 2 * (p.each * p.kpairs / p.share) : 0x7fffffff;
}

Division stream_division(int T, int K, int Nout) {
  const Plan p = plan(T, K, Nout);
  return {p.share, p.TN, p.RH, p.tiles, p.clusters * p.share};
}

medusa_status stream_launch(const Args& a, int withhold, cudaStream_t s) {
  if (!encode_fn()) return MEDUSA_ERR_CUDA;
  Plan p = plan(a.T, a.K, a.Nout);
  if (!p.share) return MEDUSA_ERR_INVALID_ARG;  // more blocks than 31 bits count, and than memory holds
  p.a = a;
  p.withhold = withhold;
  const int per = kCols >> a.glog, ng = a.K >> a.glog;
  const bool tiled = a.Nout % 16 == 0 && aligned16(a.scales) && aligned16(a.zeros);
  p.slot_bytes = p.RH * (kCols + (tiled ? 2 * per * (a.zeros ? 3 : 2) : 0));
  CUtensorMap mw, mx, ms, mz;
  if (!make_map(&mw, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.q, a.K / 2, a.Nout, a.K / 2, kCols, p.RH, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !(p.slabs == 4 ? make_slabs(&mx, a, p.TN) : make_map(&mx, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.x, a.K, a.T, a.ldx * 2, 64, p.TN, CU_TENSOR_MAP_SWIZZLE_128B)))
    return MEDUSA_ERR_CUDA;
  ms = mz = mw;
  if (tiled && (!make_map(&ms, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.scales, a.Nout, ng, (long long)a.Nout * 2, p.RH, 2 * per, CU_TENSOR_MAP_SWIZZLE_NONE) ||
                (a.zeros && !make_map(&mz, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.zeros, a.Nout, ng, a.Nout, p.RH, 2 * per, CU_TENSOR_MAP_SWIZZLE_NONE))))
    return MEDUSA_ERR_CUDA;
  auto kern = a.glog == 5 ? (tiled ? stream_kernel<4, true> : stream_kernel<4, false>)
              : a.glog == 6 ? (tiled ? stream_kernel<2, true> : stream_kernel<2, false>)
                            : (tiled ? stream_kernel<1, true> : stream_kernel<1, false>);
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem) != cudaSuccess) return MEDUSA_ERR_CUDA;
  launch_clusters(kern, p.clusters * p.share, kThreads, kSmem, p.share, s, mw, mx, ms, mz, p);
  return launch_status();
}

}  // namespace w4
}  // namespace medusa
